"""Causal attention over packed prompts (prompt_attention) on the GPU against the fp64 oracle
(oracle/prompt.py) on the same inputs.

Tolerance, from the arithmetic. With w_j the weights of a row, o its output, V the
largest |v| of its sequence:
  - the output is rounded to bf16: 2^-8 |o|;
  - the probabilities enter the product rounded to bf16 (2^-8 of each), the sum
    does not take them as rounded: 2^-8 sum_j w_j |v_j|;
  - scores: products are exact, their sum over D terms runs through D / 16
    tensor-core steps, and the scale, cap, bias and exponent are a few fp32
    operations: (D / 16 + 8) 2^-23 A <= 2^-18 A for D <= 256, with A the largest
    sum of |q_d k_d| * scale plus the largest |bias|; a cap's own rounding is
    2^-22 of it, twice. An error of e in every score moves a weighted mean by
    at most 2 e V.
What these lift above one another is the factor 1 + 2^-7.
"""
import numpy as np
import pytest
import torch

from oracle import prompt as opr

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _f(t):
    return t.detach().float().cpu().double().numpy()


def _i(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _inputs(seed, lens, Hq, Hkv, D, gaps=False):
    """(q, k, v, cu): slices of a fused projection; with gaps, rows of no sequence before and behind."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    cu = [3 if gaps else 0]
    for L in lens:
        cu.append(cu[-1] + L)
    T = cu[-1] + (5 if gaps else 0)
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device=DEV)
    qkv[:, :Hq] *= 1.5
    qkv = qkv.to(torch.bfloat16)
    return qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], cu


def _call(q, k, v, cu, expect=0, **how):
    import target_model_verify_gb300 as tv
    n = tv.prompt_attention_workspace_bytes(len(cu) - 1, *q.shape[:2], k.shape[1], q.shape[2])
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    out = tv.prompt_attention(q, k, v, _i(cu), workspace=ws, **how)
    assert tv.read_status(ws) == expect
    return out


def _check(q, k, v, cu, out, **how):
    if how.get("slopes") is not None:
        how["slopes"] = _f(how["slopes"])
    want, spread = opr.attention(_f(q), _f(k), _f(v), cu, **how)
    got = _f(out)
    D, G, scale = q.shape[2], q.shape[1] // k.shape[1], how.get("scale") or q.shape[2] ** -0.5
    for lo, hi in zip(cu, cu[1:]):
        if hi == lo:
            continue
        qq, kk, V = np.abs(_f(q[lo:hi])), np.abs(_f(k[lo:hi])), np.abs(_f(v[lo:hi])).max()
        A = max(float((qq[:, h] @ kk[:, h // G].T).max()) for h in range(q.shape[1])) * scale
        if how.get("slopes") is not None:
            A += float(np.abs(how["slopes"]).max()) * (hi - lo)
        e = 2.0 ** -18 * A + 2 * 2.0 ** -22 * how.get("softcap", 0.0)
        tol = (2.0 ** -8 * (np.abs(want[lo:hi]) + spread[lo:hi]) + 2 * e * V) * (1 + 2.0 ** -7)
        err = np.abs(got[lo:hi] - want[lo:hi])
        assert np.isfinite(got[lo:hi]).all()
        assert (err <= tol).all(), (lo, hi, float(err.max()), float((err - tol).max()))


@pytest.mark.parametrize("lens,Hq,Hkv,D", [
    ([1], 1, 1, 128),                          # one token
    ([1], 8, 2, 64),
    ([1], 2, 1, 256),
    ([300], 8, 2, 128),                        # grouped heads
    ([515], 4, 4, 64),                         # a head per group: tiles of 128 tokens
    ([333], 4, 2, 256),                        # wide heads
    ([1, 2, 0, 31, 64, 65, 127, 128, 129, 255, 256, 257], 4, 1, 128),
    ([200, 0, 0, 77], 10, 2, 128),             # five heads: tiles of 125 rows
    ([90, 140], 7, 1, 256),
    ([130], 128, 1, 64),                       # 128 heads: a token a tile
    ([40, 33], 100, 1, 128),                   # 100: rows to spare
    ([10] * 70, 16, 8, 64),                    # more items than CTAs
])
def test_matches_oracle(lens, Hq, Hkv, D):
    q, k, v, cu = _inputs(len(lens) + D, lens, Hq, Hkv, D)
    _check(q, k, v, cu, _call(q, k, v, cu))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("how", [
    {"softcap": 5.0}, {"window": 1}, {"window": 37}, {"window": 128}, {"window": 129},
    {"window": 300, "softcap": 30.0, "scale": 0.2}, {"slopes": True},
    {"slopes": True, "window": 64, "softcap": 20.0}, {"window": 2 ** 31 - 1}, {"window": 2 ** 40},
], ids=str)
def test_options(D, how):
    how = dict(how)
    if how.get("slopes"):
        how["slopes"] = torch.tensor([0.5, 0.25, 0.1, 0.01], device=DEV)
    q, k, v, cu = _inputs(D, [400, 5, 129], 4, 2, D)
    _check(q, k, v, cu, _call(q, k, v, cu, **how), **how)


@pytest.mark.parametrize("D,Hkv", [(64, 8), (128, 2), (256, 2)])
def test_a_longer_prompt(D, Hkv):
    """Many blocks that every row sees between those with masks; several items per CTA."""
    q, k, v, cu = _inputs(9, [1500, 2100], 2 * Hkv, Hkv, D)
    _check(q, k, v, cu, _call(q, k, v, cu))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_growing_scores_move_the_reference(D):
    """Later keys outweigh all before them, by more than the headroom each block."""
    q, k, v, cu = _inputs(10, [700], 2, 1, D)
    k = (k.float() * torch.linspace(0.05, 4.0, 700, device=DEV)[:, None, None]).to(torch.bfloat16)
    _check(q, k, v, cu, _call(q, k, v, cu, scale=0.5), scale=0.5)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_rows_of_no_sequence_are_left(D):
    q, k, v, cu = _inputs(11, [100, 0, 61], 4, 2, D, gaps=True)
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
    got = _call(q, k, v, cu, out=out)
    assert got is out and (out[:cu[0]] == 7).all() and (out[cu[-1]:] == 7).all()
    _check(q, k, v, cu, out)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_no_sequence_sees_another(D):
    """NaN and infinities in the rows around a sequence, and in later rows of its own."""
    q, k, v, cu = _inputs(12, [130, 200, 70], 4, 2, D)
    clean = [t.clone() for t in (q, k, v)]
    dirty = [t.clone() for t in (q, k, v)]
    for t, x in zip(dirty, (float("nan"), float("nan"), float("inf"))):
        t[:130] = x
        t[330:] = x
    for t in dirty[1:]:
        t[330 - 40:330] = float("nan")                     # the last 40 tokens' keys and values
    a, b = _call(*clean, cu), _call(*dirty, cu)
    assert torch.equal(a[130:290], b[130:290])
    assert b[290:330].isnan().all()


@pytest.mark.parametrize("D,window", [(64, 0), (128, 0), (256, 0), (128, 50)])
def test_values_that_are_no_numbers(D, window):
    """They reach the positions that see them and no others."""
    q, k, v, cu = _inputs(13, [20, 300], 4, 2, D)
    v = v.clone()
    marks = ((20 + 133, 3, float("inf")), (20 + 150, 5, float("nan")), (20 + 290, 7, -float("inf")))
    for row, col, x in marks:
        v[row, 0, col] = x
    out = _f(_call(q, k, v, cu, window=window))
    for t in range(320):
        for row, col, x in marks:
            got = out[t, :2, col]
            if row <= t and (not window or t - row < window):
                assert (np.isnan(got) if np.isnan(x) else got == x).all(), (t, row)
            else:
                assert np.isfinite(got).all(), (t, row)
    assert np.isfinite(out[:, 2:]).all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_huge_scores(D):
    """Exponents beyond 2^20, where the subtraction alone decides: the largest score takes all."""
    q, k, v, cu = _inputs(14, [200], 2, 1, D)
    out = _call((q.float() * 2 ** 40).to(torch.bfloat16), k, v, cu)
    s = np.einsum("ihd,jd->hij", _f(q), _f(k)[:, 0])
    s[:, np.triu(np.ones((200, 200), bool), 1)] = -np.inf
    want = _f(v)[s.argmax(2), 0].transpose(1, 0, 2)
    assert (_f(out) == want).all()


def test_bad_offsets_write_nothing():
    q, k, v, _ = _inputs(15, [100], 4, 2, 64)
    for cu in ([0, 50, 40, 100], [-1, 100], [0, 101], [5, 2 ** 31 - 1, 100], [50, 10]):
        out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
        _call(q, k, v, cu, expect=-1, out=out)
        assert (out == 7).all()
    _check(q, k, v, [0, 100], _call(q, k, v, [0, 100]))


def test_empty_calls():
    import target_model_verify_gb300 as tv
    q, k, v, _ = _inputs(16, [10], 4, 2, 64)
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
    tv.prompt_attention(q, k, v, _i([0]), out=out)
    _call(q, k, v, [4, 4, 4], out=out)
    assert (out == 7).all()
    assert tv.prompt_attention(q[:0], k[:0], v[:0], _i([0, 0])).shape == (0, 4, 64)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_graphs_streams_and_repeats(D):
    """Captured and replayed on other offsets; twice alike; on another stream."""
    import target_model_verify_gb300 as tv
    q, k, v, _ = _inputs(17, [500], 8, 2, D)
    cu = _i([0, 120, 120, 400, 500])
    graph = torch.cuda.CUDAGraph()
    ws = torch.empty(tv.prompt_attention_workspace_bytes(4, 500, 8, 2, D), dtype=torch.uint8, device=DEV)
    out = torch.zeros(q.shape, dtype=torch.bfloat16, device=DEV)
    with torch.cuda.graph(graph):
        tv.prompt_attention(q, k, v, cu, out=out, workspace=ws)
    for offsets in ([0, 120, 120, 400, 500], [0, 1, 2, 3, 500], [0, 250, 499, 500, 500]):
        cu.copy_(_i(offsets))
        graph.replay()
        first = out.clone()
        graph.replay()
        assert tv.read_status(ws) == 0
        assert torch.equal(first, out)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        other = tv.prompt_attention(q, k, v, cu, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(other, out)
        _check(q, k, v, offsets, out)


def test_two_graphs_share_a_workspace():
    import target_model_verify_gb300 as tv
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    graphs = []
    for D, lens in ((128, [300, 77]), (256, [5, 140]), (64, [900])):
        q, k, v, cu = _inputs(18, lens, 8, 2, D)
        want = _call(q, k, v, cu)
        out, g, offsets = torch.zeros_like(want), torch.cuda.CUDAGraph(), _i(cu)
        with torch.cuda.graph(g):
            tv.prompt_attention(q, k, v, offsets, out=out, workspace=ws)
        graphs.append((g, out, want, (q, k, v, offsets)))
    for _ in range(3):
        for g, *_ in graphs:
            g.replay()
    assert tv.read_status(ws) == 0
    for _, out, want, _ in graphs:
        assert torch.equal(out, want)


def test_two_calls_at_once():
    """On streams of their own, each with its own workspace."""
    import target_model_verify_gb300 as tv
    calls = [_inputs(19 + x, lens, 8, 2, D) for x, (D, lens) in enumerate(((128, [2000]), (64, [300] * 5), (256, [700])))]
    want = [_call(*c) for c in calls]
    offsets = [_i(c[3]) for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        outs = [tv.prompt_attention(*c[:3], cu, stream=s) for c, cu, s in zip(calls, offsets, streams)]
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


def test_many_short_sequences():
    """More sequences than threads of the kernel that lists the work, empty ones among them."""
    lens = [(7 * x) % 5 for x in range(3000)]
    q, k, v, cu = _inputs(23, lens, 4, 2, 64)
    _check(q, k, v, cu, _call(q, k, v, cu))
