"""Causal attention over packed prompts, in fp64.

Test infrastructure only (see the package docstring): written from the
definitions in include/specdec_verify.h, sharing no code with the library.
"""
from __future__ import annotations

import math

import numpy as np


def attention(q, k, v, cu_seqlens, scale=0.0, softcap=0.0, window=0, slopes=None):
    """(out [T, Hq, D], spread [T, Hq, D]): the outputs, and sum_j w_j |v_j|; NaN in rows of no sequence."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    scale = scale if scale > 0 else 1.0 / math.sqrt(D)
    out, spread = np.full((T, Hq, D), np.nan), np.full((T, Hq, D), np.nan)
    for lo, hi in zip(cu_seqlens, cu_seqlens[1:]):
        L = hi - lo
        if L == 0:
            continue
        away = np.arange(L)[:, None] - np.arange(L)[None, :]
        see = away >= 0
        if window:
            see &= away < window
        for h in range(Hq):
            s = scale * (q[lo:hi, h] @ k[lo:hi, h // G].T)
            if softcap:
                s = softcap * np.tanh(s / softcap)
            if slopes is not None:
                s = s - float(slopes[h]) * away
            s = np.where(see, s, -np.inf)
            e = np.exp(s - s.max(1, keepdims=True))
            w = e / e.sum(1, keepdims=True)
            out[lo:hi, h] = w @ v[lo:hi, h // G]
            spread[lo:hi, h] = w @ np.abs(v[lo:hi, h // G])
    return out, spread
