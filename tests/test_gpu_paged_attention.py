"""Attention over a paged bf16 cache (verify_attention_paged) on the GPU: against the fp64 oracle with the
tolerances of tests/test_gpu_cache_attention.py (the arithmetic is the masked attention's), and, for more
query rows than the form for little work takes, bit for bit against the masked attention of the same rows
laid end to end."""
import numpy as np
import pytest
import torch

from oracle import cache as oc
from oracle import paged as op
from tests.test_gpu_cache_attention import TREE26, _check, _f

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _i(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _inputs(seed, B, n, Hq, Hkv, D, page, max_pages, lens, spare=3):
    """Pages in any order; what belongs to no sequence holds NaN, and so do the rows behind a sequence's end."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    q = (torch.randn(B, n, Hq, D, generator=g, device=DEV) * 1.5).to(torch.bfloat16)
    held = [-(-L // page) for L in lens]
    total = sum(held) + spare
    order = torch.randperm(total, generator=g, device=DEV).tolist()
    pages = [torch.randn(total, page, Hkv, D, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2)]
    table, at = [[-1] * max_pages for _ in range(B)], 0
    for b, h in enumerate(held):
        table[b][:h] = order[at:at + h]
        at += h
        if lens[b] % page:
            for t in pages:
                t[table[b][h - 1], lens[b] % page:] = float("nan")
    for t in pages:
        t[order[at:]] = float("nan")
    return q, pages, _i(table), _i(lens)


def _flat(pages, table, lens, Lmax):
    """The sequences' rows end to end, [B, Lmax, Hkv, D]; zeros behind them."""
    out = []
    for t in pages:
        c = torch.zeros(len(lens), Lmax, *t.shape[2:], dtype=t.dtype, device=DEV)
        for b, L in enumerate(lens.tolist()):
            ids = table[b, :-(-L // t.shape[1])].long()
            c[b, :L] = t[ids].flatten(0, 1)[:L]
        out.append(c)
    return tuple(out)


def _call(q, pages, table, lens, expect=0, **how):
    import target_model_verify_gb300 as tv
    B, n, Hq, D = q.shape
    ws = torch.empty(tv.paged_attention_workspace_bytes(B, n, Hq, pages[0].shape[2], D, *pages[0].shape[:2],
                                                        table.shape[1]), dtype=torch.uint8, device=DEV)
    out = tv.verify_attention_paged(q, *pages, table, lens, workspace=ws, **how)
    assert tv.read_status(ws) == expect
    return out


def _run(q, pages, table, lens, **how):
    import target_model_verify_gb300 as tv
    out = _call(q, pages, table, lens, **how)
    flat = _flat(pages, table, lens, table.shape[1] * pages[0].shape[1])
    if q.shape[1] * q.shape[2] // pages[0].shape[2] > 16:
        assert torch.equal(out, tv.verify_attention_masked(q, *flat, lens, **how))
    _check("masked", q, flat, lens, out, **how)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("n,Hq,Hkv,D", [
    (1, 1, 1, 128),               # one head
    (1, 32, 8, 128),              # a drafter's token, Llama grouping
    (5, 8, 2, 64),
    (3, 4, 4, 256),               # wide heads, no grouping
    (9, 16, 2, 128),              # 72 rows: two groups
    (40, 2, 2, 64),               # 64 lanes of rows
])
def test_matches_oracle_and_masked(page, n, Hq, Hkv, D):
    lens = [n, 0, n + 15, n + 16, n + 17, 127, 128, 129, 300, 511]
    q, pages, table, lens = _inputs(page + D, len(lens), n, Hq, Hkv, D, page, 512 // page + 1, lens)
    _run(q, pages, table, lens)


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("how", [
    {"softcap": 5.0}, {"window": 1}, {"window": 37}, {"window": 200, "softcap": 30.0, "scale": 0.2},
    {"slopes": True}, {"slopes": True, "window": 64, "softcap": 20.0},
    {"parent": TREE26}, {"parent": TREE26, "window": 3}, {"parent": TREE26, "slopes": True, "softcap": 10.0},
], ids=str)
def test_options(page, D, how):
    n = 26 if "parent" in how else 4
    how = dict(how)
    if how.get("slopes"):
        how["slopes"] = torch.tensor([0.5, 0.25, 0.1, 0.01], device=DEV)
    q, pages, table, lens = _inputs(D + n, 3, n, 4, 2, D, page, 320 // page, [310, n, 129])
    _run(q, pages, table, lens, **how)


@pytest.mark.parametrize("page", [16, 128])
def test_one_long_sequence_and_many_short_ones(page):
    q, pages, table, lens = _inputs(1, 1, 1, 8, 2, 128, page, 20000 // page + 1, [19999])
    _run(q, pages, table, lens)
    many = [1 + 37 * b % 500 for b in range(70)]
    q, pages, table, lens = _inputs(2, 70, 1, 16, 8, 64, page, 512 // page, many)
    _run(q, pages, table, lens)


# 2 query heads per KV head: up to 8 new positions go to the form for little work, 9 to the other
FORMS = pytest.mark.parametrize("n", [3, 9])


@FORMS
def test_pages_behind_the_window_may_be_gone(n):
    """What no position sees is not looked up: entries of pages given back hold anything."""
    q, pages, table, lens = _inputs(3, 2, n, 4, 2, 128, 16, 70, [1100, 600])
    want = _call(q, pages, table, lens, window=100)
    gone = table.clone()
    gone[0, :(1100 - n - 100 + 1) // 16] = -1
    gone[1, :(600 - n - 100 + 1) // 16] = 1 << 30
    assert torch.equal(_call(q, pages, gone, lens, window=100), want)
    gone[1, (600 - n - 100 + 1) // 16] = -1
    _call(q, pages, gone, lens, window=100, expect=op.INVALID)


@FORMS
@pytest.mark.parametrize("D", [64, 128, 256])
def test_pages_outside_the_pool_count_as_zeros(n, D):
    for bad in (-1, 1 << 30, 2 ** 31 - 1, -2 ** 31):
        q, pages, table, lens = _inputs(4, 2, n, 4, 2, D, 16, 20, [310, 200])
        if bad == 1 << 30:
            bad = pages[0].shape[0]                      # the first that there is not
        table[0, 4] = table[1, 12] = table[0, 19] = bad
        out = _call(q, pages, table, lens, expect=op.INVALID)
        host = table.tolist()
        k, v = (np.stack([np.pad(op.gather(_f(t), host[b], L), ((0, 320 - L), (0, 0), (0, 0)))
                          for b, L in enumerate((310, 200))]) for t in pages)
        want = oc.masked_attention(_f(q), k, v, [310, 200])
        # the output's rounding, the weights', and the scores' well within it
        assert (np.abs(_f(out) - want) <= 2.0 ** -8 * np.abs(want) + 3 * 2.0 ** -8 * np.abs(v).max()).all()
        table[0, 4] = table[1, 12] = table[0, 19] = 0
        _call(q, pages, table, lens)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,Hq", [(4, 4), (4, 12)])           # 8 rows, 24 rows
def test_values_that_are_no_numbers(n, Hq, D):
    """They reach the positions that see them and no others, found through the table."""
    q, pages, table, lens = _inputs(5, 1, n, Hq, 2, D, 16, 10, [150])
    for row, col, x in ((147, 3, float("inf")), (148, 5, float("nan")), (149, 7, -float("inf"))):
        pages[1][table[0, row // 16], row % 16, 0, col] = x
    out = _f(_call(q, pages, table, lens))[0]
    for i in range(4):
        for row, col, x in ((147, 3, np.inf), (148, 5, np.nan), (149, 7, -np.inf)):
            for h in range(Hq // 2):
                got = out[i, h, col]
                if row <= 146 + i:
                    assert np.isnan(got) if np.isnan(x) else got == x
                else:
                    assert np.isfinite(got)
            assert np.isfinite(out[i, Hq // 2:, col]).all()


@FORMS
def test_bad_lengths(n):
    q, pages, table, lens = _inputs(6, 4, n, 4, 2, 64, 16, 4, [64, 30, 20, 33])
    good = _call(q, pages, table, lens)
    out = _call(q, pages, table, _i([65, -1, n - 1, 33]), expect=op.INVALID)
    assert not out[:3].any() and torch.equal(out[3], good[3])


@pytest.mark.parametrize("n", [2, 5])                        # 8 rows, 20 rows
def test_strided_queries_streams_and_graphs(n):
    import target_model_verify_gb300 as tv
    q, pages, table, lens = _inputs(7, 3, n, 8, 2, 128, 32, 12, [300, n, 77])
    want = _call(q, pages, table, lens)
    wide = torch.randn(3, n, 12, 128, device=DEV).to(torch.bfloat16)
    wide[:, :, :8] = q
    assert torch.equal(_call(wide[:, :, :8], pages, table, lens), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = tv.verify_attention_paged(q, *pages, table, lens, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = tv.verify_attention_paged(q, *pages, table, lens)
    for _ in range(2):
        q.copy_(q.flip(1))
        lens.copy_(lens.roll(1))
        table.copy_(table.roll(1, 0))
        graph.replay()
        assert torch.equal(out, _call(q, pages, table, lens))


@pytest.mark.parametrize("B,n,Hq,Hkv,D,capacity,lens", [
    (1, 1, 4, 1, 128, 8192, [8192]),             # eight CTAs, eight chunks a warp
    (1, 16, 1, 1, 64, 8192, [8000]),             # sixteen positions of one head
    (18, 1, 16, 8, 128, 1024, None),             # a CTA to a tile, the most tiles at once less a few
    (9, 1, 16, 8, 128, 2048, None),              # two
    (4, 1, 16, 8, 128, 4096, None),              # four
    (50, 2, 18, 9, 64, 256, None),               # 64 dims: three CTAs to an SM
    (2, 3, 10, 2, 256, 2048, [2048, 3]),
    (37, 1, 4, 4, 256, 256, None),
])
@pytest.mark.parametrize("how", [{}, {"window": 77}, {"slopes": True, "softcap": 20.0}], ids=str)
def test_little_work(B, n, Hq, Hkv, D, capacity, lens, how):
    """The form for little work at each size of its clusters, up to the longest that it takes."""
    how = dict(how)
    if how.get("slopes"):
        how["slopes"] = torch.exp2(-torch.arange(1, Hq + 1, device=DEV, dtype=torch.float32))
    if lens is None:
        lens = [n + 131 * b % (capacity - n) for b in range(B)]
        lens[0] = capacity
    q, pages, table, lens = _inputs(B + D, B, n, Hq, Hkv, D, 16, capacity // 16, lens)
    _run(q, pages, table, lens, **how)


@pytest.mark.parametrize("n,parent", [(1, False), (8, False), (26, True)])
def test_small_trees_and_lengths(n, parent):
    """Every length from the new positions' count on, across the first chunks' edges."""
    lens = list(range(n, n + 36))
    q, pages, table, lens = _inputs(8, len(lens), n, 2, 2, 128, 16, 5, lens)
    _run(q, pages, table, lens, **({"parent": TREE26[:n]} if parent else {}))


def test_a_small_tree_in_the_form_for_little_work():
    for how in ({}, {"window": 3}, {"slopes": torch.tensor([0.5, 0.1], device=DEV)}):
        q, pages, table, lens = _inputs(9, 4, 14, 2, 2, 128, 32, 5, [14, 31, 60, 137])
        _run(q, pages, table, lens, parent=TREE26[:14], **how)


def test_two_graphs_share_a_workspace():
    """Steps of two layers, captured apart with one workspace, replayed in turn."""
    import target_model_verify_gb300 as tv
    graphs, outs, wants = [], [], []
    ws = torch.empty(1 << 26, dtype=torch.uint8, device=DEV)
    for layer, n in ((0, 1), (1, 9)):
        q, pages, table, lens = _inputs(20 + layer, 3, n, 8, 2, 128, 16, 40, [600, 77, 300])
        wants.append(_call(q, pages, table, lens))
        out, g = torch.zeros_like(q), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            tv.verify_attention_paged(q, *pages, table, lens, out=out, workspace=ws)
        graphs.append((g, q, pages, table, lens))
        outs.append(out)
    for _ in range(3):
        for g, *_ in graphs:
            g.replay()
    assert tv.read_status(ws) == 0
    for out, want in zip(outs, wants):
        assert torch.equal(out, want)


def test_two_calls_at_once():
    """On streams of their own, each with its own workspace."""
    import target_model_verify_gb300 as tv
    calls = [_inputs(30, 2, n, 8, 2, 128, 16, 300, [4000, 900]) for n in (1, 1, 9, 9)]
    want = [_call(*c) for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        outs = [tv.verify_attention_paged(c[0], *c[1], c[2], c[3], stream=s) for c, s in zip(calls, streams)]
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
