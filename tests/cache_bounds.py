"""How far the cache attention may be from the formula, output by output (fp64, numpy).

For one sequence, with w_j the softmax weights of a query row, o its output, s_j
the scale of value row j (1 over a bf16 cache) and c_j = v_j / s_j:

  - the output is rounded to bf16: 2^-8 |o|;
  - masked: a weight is rounded to bf16, and the sum takes it as rounded, so o
    moves by at most 2^-8 sum_j w_j |v_j - o|;
  - kv8: a weight is rounded to f16, 2^-11 of it, and below f16's normal numbers
    to a fixed step, half of which is at most 2^-32 of the largest w_j s_j, and
    at most 2^-11 of the largest among the cache rows that share a reference in
    one block, no more than 128 (or those are below 2^-45 of the largest of
    all). The sum is not rounded. Together 2^-11 sum_j w_j |v_j| +
    sum_j max(min(2^-11 max_block(w s), 2^-32 max(w s)), 2^-45 max(w s)) |c_j|;
  - an error of at most e in every score moves o by at most
    e sum_j w_j |v_j - o| (to first order; e^2 of that is left to the slack).
    e: the product's sum over D terms runs through D / 16 tensor-core steps,
    scale, cap, bias and exponent are a few fp32 operations, in all
    (D / 16 + 8) 2^-23 A <= 2^-18 A for D <= 256, with A the largest
    scale * sum_d |q_d k_jd| plus the largest |bias|; a cap's own rounding is
    2^-22 of the cap, twice; kv8 queries are two e4m3 terms of the row scaled
    to a largest element in [2^7, 2^8), so each element is off by at most half
    of the second term's last step, 2^-10, or 2^-17 of the largest:
    2^-17 max_d |q_d| * scale * max_j sum_d |k_jd|.

Nothing of this grows with the length.
"""
import math

import numpy as np

BLOCK = 128


def sight(n, L, window=0, parent=None):
    """(which of L rows position i sees [n, L], their distances [n, L])."""
    P = L - n
    parent = list(range(-1, n - 1)) if parent is None else list(parent)
    depth = [0] * n
    see = np.zeros((n, L), dtype=bool)
    see[:, :P] = True
    for i in range(n):
        a = i
        while a >= 0:
            see[i, P + a] = True
            a = parent[a]
        depth[i] = 0 if i == 0 else depth[parent[i]] + 1
    pos = np.concatenate([np.arange(P), P + np.array(depth)])
    away = (P + np.array(depth))[:, None] - pos[None, :]
    if window:
        see &= away < window
    return see, away


def outputs_and_bounds(kind, q, k, v, sv=None, scale=0.0, softcap=0.0, window=0, slopes=None, parent=None,
                       without=0):
    """(o, bound), each [n, Hq, D], of one sequence: q [n, Hq, D], k and v [L, Hkv, D], sv [L, Hkv].

    without: also [blocks]: for every run of that many rows, how many times its bound some output
    moves when the run is left out (what a lost partial would do).
    """
    n, Hq, D = q.shape
    L, Hkv, _ = k.shape
    G = Hq // Hkv
    scale = scale if scale > 0 else 1.0 / math.sqrt(D)
    see, away = sight(n, L, window, parent)
    sv = np.ones((L, Hkv)) if sv is None else sv
    out, tol = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    edges = np.arange(0, L, BLOCK)
    shows = np.zeros(-(-L // without)) if without else None
    for h in range(Hq):
        kk, vv, ss = k[:, h // G], v[:, h // G], sv[:, h // G]
        s = scale * (q[:, h] @ kk.T)
        A = scale * (np.abs(q[:, h]) @ np.abs(kk).T).max(1)
        if softcap:
            s = softcap * np.tanh(s / softcap)
        if slopes is not None:
            s = s - float(slopes[h]) * away
            A = A + abs(float(slopes[h])) * np.abs(away * see).max(1)
        s = np.where(see, s, -np.inf)
        w = np.exp(s - s.max(1, keepdims=True))
        w /= w.sum(1, keepdims=True)
        o = w @ vv
        e = 2.0 ** -18 * A + 2 * 2.0 ** -22 * softcap
        if kind != "masked":
            e = e + 2.0 ** -17 * np.abs(q[:, h]).max(1) * scale * np.abs(kk).sum(1).max()
        for i in range(n):
            spread = w[i] @ np.abs(vv - o[i])
            t = 2.0 ** -8 * np.abs(o[i]) + e[i] * (1 + 2 * e[i]) * spread
            if kind == "masked":
                t = t + 2.0 ** -8 * spread
            else:
                top = np.repeat(np.maximum.reduceat(w[i] * ss, edges), BLOCK)[:L]
                step = np.maximum(np.minimum(2.0 ** -11 * top, 2.0 ** -32 * top.max()), 2.0 ** -45 * top.max())
                t = t + 2.0 ** -11 * (w[i] @ np.abs(vv)) + (step * see[i] / ss) @ np.abs(vv)
            tol[i, h] = t * (1 + 2.0 ** -7)          # products of the above, and of them with the bf16 rounding
            if without:
                runs = np.arange(0, L, without)
                lost = np.add.reduceat(w[i][:, None] * vv, runs)                   # [blocks, D]
                share = np.add.reduceat(w[i], runs)[:, None]
                moved = np.abs((o[i] - lost) / np.maximum(1 - share, 1e-30) - o[i])
                shows = np.maximum(shows, (moved / tol[i, h]).max(1))
        out[:, h] = o
    return (out, tol, shows) if without else (out, tol)


# ------------------------------------------------------------------ inputs --

def with_sink(rng, n, Hq, Hkv, D, L, weight, sigma=1.0):
    """q, k, v [.., D] of a sequence whose first row takes about `weight` of every position, with value 0:
    dim 0 of the queries and of that key is theirs alone. The values have a mean per channel."""
    q = rng.standard_normal((n, Hq, D)) * sigma
    k = rng.standard_normal((L, Hkv, D))
    v = np.sign(rng.standard_normal((1, Hkv, D))) + 0.5 * rng.standard_normal((L, Hkv, D))
    rest = math.log(L) + sigma ** 2 / 2
    q[:, :, 0], k[:, :, 0] = 8.0, 0.0
    k[0] = 0.0
    k[0, :, 0] = (rest + math.log(weight / (1 - weight))) * math.sqrt(D) / 8.0
    v[0] = 0.0
    return q, k, v


def with_marks(rng, n, Hq, Hkv, D, L, block=64):
    """q, k, v of a sequence in which every `block` rows have a dim whose values are theirs (24 on
    top of noise), so that each run of them shows in the output."""
    q = rng.standard_normal((n, Hq, D)) * 0.5
    k = rng.standard_normal((L, Hkv, D))
    v = 0.25 * rng.standard_normal((L, Hkv, D))
    at = np.arange(L)
    v[at, :, (at // block) % D] += 24.0
    return q, k, v
