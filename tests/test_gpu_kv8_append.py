"""Appending to the 8-bit cache on the GPU (append_kv8) against the fp64 oracle
(oracle/cache.py).

Scales are powers of two, so x / scale is exact and every code and scale has
one right value: the comparisons are for equality.
"""
import numpy as np
import pytest
import torch

from oracle import cache as oc

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _cache(g, B, Lmax, H, D):
    """A filled cache: random codes (no NaN) and power-of-two scales."""
    def one():
        codes = (torch.randn(B, Lmax, H, D, generator=g, device=DEV) * 60).clamp(-448, 448)
        e = torch.randint(-9, -5, (B, H, -(-Lmax // 32)), generator=g, device=DEV)
        return codes.to(torch.float8_e4m3fn), torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)
    (k, ks), (v, vs) = one(), one()
    return k, v, ks, vs


def _f(t):
    return t.detach().float().cpu().double().numpy()


def _i(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _run_and_check(new, cache, start, counts=None, rows=None):
    import target_model_verify_gb300 as tv
    want = [oc.append(_f(new[0]), _f(cache[0]), _f(cache[2]), start, counts, rows),
            oc.append(_f(new[1]), _f(cache[1]), _f(cache[3]), start, counts, rows)]
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    tv.append_kv8(*new, *cache, _i(start), None if counts is None else _i(counts),
                  None if rows is None else _i(rows), workspace=ws)
    assert tv.read_status(ws) == 0
    for x, (codes, scales) in ((0, want[0]), (1, want[1])):
        np.testing.assert_array_equal(_f(cache[2 + x]), scales)
        np.testing.assert_array_equal(_f(cache[x]), codes)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,n,H,Lmax,start", [
    (1, 1, 1, 1, [0]),                    # a cache of one row
    (3, 5, 8, 100, [0, 30, 95]),          # first row, across a block's edge, to the cache's end
    (2, 33, 3, 97, [31, 64]),             # three blocks, a ragged last one
    (1, 70, 2, 200, [32]),                # whole blocks
])
def test_append_matches_oracle(D, B, n, H, Lmax, start):
    g = torch.Generator(device=DEV).manual_seed(D + n)
    new = [(torch.randn(B, n, H, D, generator=g, device=DEV) * 3).to(torch.bfloat16) for _ in range(2)]
    _run_and_check(new, _cache(g, B, Lmax, H, D), start)


def test_growing_scale_encodes_earlier_rows_again():
    """New rows of 40 times the block's magnitude, and of 1/40 of it."""
    g = torch.Generator(device=DEV).manual_seed(3)
    for factor in (40.0, 1 / 40.0):
        cache = _cache(g, 2, 64, 2, 128)
        new = [(torch.randn(2, 3, 2, 128, generator=g, device=DEV) * factor).to(torch.bfloat16)
               for _ in range(2)]
        _run_and_check(new, cache, [29, 50])


def test_slices_counts_and_rows():
    """A fused projection's slices, ragged counts, rows picked from a tree's (one twice)."""
    g = torch.Generator(device=DEV).manual_seed(4)
    B, n, H, D = 4, 7, 2, 128
    kv = torch.randn(B, n, 2, H, D, generator=g, device=DEV).to(torch.bfloat16)
    new = [kv[:, :, 0], kv[:, :, 1]]
    _run_and_check(new, _cache(g, B, 90, H, D), [0, 31, 60, 83], counts=[7, 0, 1, -1])
    rows = [[0, 2, 5, -1, -1, -1, -1], [6, -1, -1, -1, -1, -1, -1], [1, 1, 3, 4, 5, 6, 0], [-1] * 7]
    _run_and_check(new, _cache(g, B, 90, H, D), [5, 31, 62, 90], counts=[3, 1, 7, 0], rows=rows)
    one = kv[:, :1]                       # one position per sequence: the sequences' stride counts
    _run_and_check([one[:, :, 0], one[:, :, 1]], _cache(g, B, 90, H, D), [0, 31, 32, 89])


def test_extreme_values():
    """Zeros, the scale's clamps, values on the border of a scale, infinities and NaN."""
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.zeros(1, 8, 8, 64, device=DEV)
    x[:, :, 1] = 448.0                     # fits scale 1 exactly
    x[:, :, 2] = 450.0                     # the next bf16: scale 2
    x[:, :, 3] = 1e-30                     # below the smallest scale's reach
    x[:, :, 4] = 3e38                      # above the largest scale's
    x[:, :, 5] = torch.randn(64, generator=g, device=DEV)
    x[:, 2, 5, 3], x[:, 3, 5, 4], x[:, 4, 5, 5] = float("inf"), -float("inf"), float("nan")
    x[:, :, 6] = float("nan")
    x[:, :, 7] = torch.linspace(-300, 300, 64, device=DEV)
    x = x.to(torch.bfloat16)
    _run_and_check([x, -x], _cache(g, 1, 40, 8, 64), [30])


def test_rows_outside_are_left():
    """Only the new rows' codes and their blocks' scales change."""
    import target_model_verify_gb300 as tv
    g = torch.Generator(device=DEV).manual_seed(6)
    cache = _cache(g, 2, 128, 2, 128)
    before = [t.view(torch.uint8).clone() for t in cache]
    new = [torch.randn(2, 4, 2, 128, generator=g, device=DEV).to(torch.bfloat16) * 1e-6 for _ in range(2)]
    tv.append_kv8(*new, *cache, _i([10, 64]))          # small: no scale grows in a shared block
    for was, now in zip(before[:2], cache[:2]):
        now = now.view(torch.uint8)
        keep = torch.ones(2, 128, dtype=torch.bool, device=DEV)
        keep[0, 10:14] = keep[1, 64:68] = False
        assert torch.equal(was[keep], now[keep])
    for was, now in zip(before[2:], cache[2:]):
        keep = torch.ones(2, 2, 4, dtype=torch.bool, device=DEV)
        keep[1, :, 2] = False
        assert torch.equal(was.view(torch.float32)[keep], now[keep])


def test_bad_tables_set_the_status_and_skip():
    import target_model_verify_gb300 as tv
    g = torch.Generator(device=DEV).manual_seed(7)
    B, n, H, D = 5, 4, 1, 64
    new = [torch.randn(B, n, H, D, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2)]
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    for start, counts, rows, bad in (
            ([0, -1, 61, 3, 2 ** 31 - 1], None, None, [1, 2, 4]),
            ([0, 0, 0, 0, 0], [4, 5, 2 ** 31 - 1, 0, -7], None, [1, 2]),
            ([0, 0, 0, 0, 0], [2, 2, 1, 0, 4], [[0, 1, 9, 9], [0, 4, 0, 0], [-1, 0, 0, 0], [7, 7, 7, 7],
                                               [3, 2, 1, 0]], [1, 2])):
        cache = _cache(g, B, 64, H, D)
        before = [t.view(torch.uint8).clone() for t in cache]
        tv.append_kv8(*new, *cache, _i(start), None if counts is None else _i(counts),
                      None if rows is None else _i(rows), workspace=ws)
        assert tv.read_status(ws) == tv._b.SPECDEC_ERR_INVALID_ARG
        for was, now in zip(before, cache):
            for b in bad:
                assert torch.equal(was[b], now.view(torch.uint8)[b])
        for was, now in zip(before[:2], cache[:2]):       # (a scale may come out as it was)
            assert not torch.equal(was[0], now.view(torch.uint8)[0])
    tv.append_kv8(*new, *cache, _i([0] * 5), workspace=ws)
    assert tv.read_status(ws) == 0


def test_captured_append():
    import target_model_verify_gb300 as tv
    g = torch.Generator(device=DEV).manual_seed(8)
    new = [torch.randn(2, 3, 2, 128, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2)]
    cache, start = _cache(g, 2, 64, 2, 128), _i([0, 5])
    other = [t.clone() for t in cache]
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        tv.append_kv8(*new, *cache, start, workspace=ws)
    start += 3
    graph.replay()
    tv.append_kv8(*new, *other, start)
    torch.cuda.synchronize()
    for a, b in zip(cache, other):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
