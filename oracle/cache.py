"""The 8-bit key/value cache and the masked verify-step attention, in fp64.

Test infrastructure only (see the package docstring): written from the
definitions in include/specdec_verify.h, sharing no code with the library.

Codes are e4m3 values (1 sign, 4 exponent, 3 mantissa bits, bias 7, largest
448, one NaN); a cache is a float array of those values [B, Lmax, Hkv, D] with
scales [B, Hkv, ceil(Lmax / 32)].
"""
from __future__ import annotations

import math

import numpy as np

BLOCK = 32


def e4m3_values() -> np.ndarray:
    """The 127 non-negative finite e4m3 values in code order."""
    out = []
    for code in range(127):
        e, m = code >> 3, code & 7
        out.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return np.array(out)


_VALUES = e4m3_values()


def to_e4m3(x) -> np.ndarray:
    """Nearest e4m3 value, ties to the even code, saturating; NaN stays."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.minimum(np.searchsorted(_VALUES, np.nan_to_num(a, nan=0.0), side="left"), 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _VALUES[lo], _VALUES[hi] - a
    pick = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return np.where(np.isnan(x), np.nan, np.copysign(_VALUES[pick], x))


def block_scale(amax: float) -> float:
    """The smallest 2^e, e in [-40, 40], with amax <= 448 * 2^e (2^-40 for 0)."""
    for e in range(-40, 40):
        if amax <= math.ldexp(448.0, e):
            return math.ldexp(1.0, e)
    return math.ldexp(1.0, 40)


def append(new, codes, scales, start, counts=None, rows=None):
    """Copies of (codes, scales) with new [B, n, H, D] written from row start[b] on."""
    new = np.asarray(new, dtype=np.float64)
    codes, scales = np.array(codes, dtype=np.float64), np.array(scales, dtype=np.float64)
    B, n, H, _ = new.shape
    for b in range(B):
        c = n if counts is None else int(counts[b])
        s0 = int(start[b])
        if c <= 0:
            continue
        for h in range(H):
            for blk in range(s0 // BLOCK, (s0 + c - 1) // BLOCK + 1):
                at = [r for r in range(blk * BLOCK, (blk + 1) * BLOCK) if s0 <= r < s0 + c]
                src = [r - s0 if rows is None else int(rows[b][r - s0]) for r in at]
                x = new[b, src, h]
                fin = np.abs(x[np.isfinite(x)])
                s = block_scale(float(fin.max()) if fin.size else 0.0)
                if blk * BLOCK < s0:
                    was = scales[b, h, blk]
                    s = max(s, was)
                    old = slice(blk * BLOCK, s0)
                    codes[b, old, h] = to_e4m3(codes[b, old, h] * (was / s))
                codes[b, at, h] = to_e4m3(x / s)
                scales[b, h, blk] = s
    return codes, scales


def dequantise(codes, scales) -> np.ndarray:
    """The values a cache stands for, [B, Lmax, Hkv, D]."""
    codes, scales = np.asarray(codes, dtype=np.float64), np.asarray(scales, dtype=np.float64)
    at = np.arange(codes.shape[1]) // BLOCK
    return codes * scales.transpose(0, 2, 1)[:, at][..., None]


def masked_attention(q, k, v, seq_lens, scale=0.0, softcap=0.0, window=0, slopes=None, parent=None):
    """fp64 attention of the new positions; 0 for sequences of length 0."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    B, n, Hq, D = q.shape
    G = Hq // k.shape[2]
    scale = scale if scale > 0 else 1.0 / math.sqrt(D)
    parent = list(range(-1, n - 1)) if parent is None else list(parent)
    out = np.zeros((B, n, Hq, D))
    for b in range(B):
        L = int(seq_lens[b])
        if L == 0:
            continue
        P = L - n
        for i in range(n):
            path = [i]
            while parent[path[-1]] >= 0:
                path.append(parent[path[-1]])
            path.reverse()                                   # root .. i
            rows = list(range(P)) + [P + a for a in path]
            pos = list(range(P)) + [P + d for d in range(len(path))]
            if window:
                keep = [x for x in range(len(rows)) if pos[-1] - pos[x] < window]
                rows, pos = [rows[x] for x in keep], [pos[x] for x in keep]
            away = pos[-1] - np.array(pos, dtype=np.float64)
            for h in range(Hq):
                s = scale * (k[b, rows, h // G] @ q[b, i, h])
                if softcap:
                    s = softcap * np.tanh(s / softcap)
                if slopes is not None:
                    s = s - float(slopes[h]) * away
                e = np.exp(s - s.max())
                out[b, i, h] = (e / e.sum()) @ v[b, rows, h // G]
    return out
