"""Attention over the 8-bit cache (verify_attention_kv8) and masked attention over a
bf16 cache (verify_attention_masked) on the GPU against the fp64 oracle
(oracle/cache.py) on the same inputs.

Tolerance, from the arithmetic. With u = finfo.eps / 2 (bf16 2^-8, f16
2^-11), V the largest visible |v| and o the output:
  - the output is rounded to bf16: 2^-8 |o|;
  - the probabilities are rounded. Over the 8-bit cache to f16, which moves a
    weighted mean of values by at most 2^-11 V; the form for many tiles then
    writes them as three e4m3 terms, exact but for the last term's half step,
    2^-10 / 256, where a row's largest probability is at least 2^2: each of L
    weights is off by at most 2^-20 of that one, the mean by 2^-20 L V (the
    row form's f16 ends at 2^-25 / 2^7 of it, 2^-32 L V). Over the bf16 cache
    to bf16, whose rounded weights are also what the sum counts, so the mean moves by
    at most 2^-8 * sum w |v - o| <= 2^-8 * 2 V;
  - scores: products are exact, their sum over D terms runs through D / 16
    tensor-core steps, and the scale, cap, bias and exponent are a few fp32
    operations: (D / 16 + 8) * 2^-23 * A <= 2^-18 A for D <= 256, with A the
    largest sum of |q_d k_d| * scale plus |bias| (the cap's own rounding,
    2^-22 of the cap, twice); an error e of the scores moves the mean by at
    most 2 e V.
"""
import numpy as np
import pytest
import torch

from oracle import cache as oc

pytestmark = pytest.mark.gpu
DEV = "cuda"
TREE26 = (-1, 0, 0, 0, 0, 1, 1, 1, 2, 2, 3, 4, 5, 5, 6, 7, 8, 10, 11, 12, 12, 13, 14, 16, 19, 21)


def _f(t):
    return t.detach().float().cpu().double().numpy()


def _inputs(kind, seed, B, n, Hq, Hkv, D, Lmax, lens=None, spread=True):
    g = torch.Generator(device=DEV).manual_seed(seed)
    q = (torch.randn(B, n, Hq, D, generator=g, device=DEV) * 1.5).to(torch.bfloat16)
    if kind != "masked":
        def one():
            c = (torch.randn(B, Lmax, Hkv, D, generator=g, device=DEV) * 60).to(torch.float8_e4m3fn)
            e = torch.randint(-7, -4, (B, Hkv, -(-Lmax // 32)), generator=g, device=DEV) if spread else \
                torch.full((B, Hkv, -(-Lmax // 32)), -6, device=DEV)
            return c, torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)
        (k, ks), (v, vs) = one(), one()
        cache = (k, v, ks, vs)
    else:
        cache = tuple(torch.randn(B, Lmax, Hkv, D, generator=g, device=DEV).to(torch.bfloat16)
                      for _ in range(2))
    if lens is None:
        lens = torch.randint(n, Lmax + 1, (B,), generator=g, device=DEV).tolist()
    return q, cache, torch.tensor(lens, dtype=torch.int32, device=DEV)


def _values(cache):
    if len(cache) == 4:
        return oc.dequantise(_f(cache[0]), _f(cache[2])), oc.dequantise(_f(cache[1]), _f(cache[3]))
    return _f(cache[0]), _f(cache[1])


def _call(kind, q, cache, lens, workspace=None, **how):
    """The call; unless the caller brings a workspace, no device-side error is expected of it."""
    import target_model_verify_gb300 as tv
    if kind == "kv8_keys":
        B, more = q.shape[0], max(0, 256 // cache[0].shape[2] + 1 - q.shape[0])
        pad = lambda t: torch.cat([t, t[:1].expand(more, *t.shape[1:])]) if t.element_size() > 1 else \
            torch.cat([t.view(torch.uint8), t[:1].view(torch.uint8).expand(more, *t.shape[1:])]).view(t.dtype)  # noqa: E731
        lens = torch.cat([lens, torch.zeros(more, dtype=torch.int32, device=DEV)])
        out, how["out"] = how.get("out"), None
        got = _call("kv8", pad(q), tuple(pad(t) for t in cache), lens, workspace=workspace, **how)
        assert not got[B:].any()
        return got[:B] if out is None else out.copy_(got[:B])
    fn = tv.verify_attention_kv8 if kind == "kv8" else tv.verify_attention_masked
    if workspace is not None or torch.cuda.is_current_stream_capturing() or "stream" in how:
        return fn(q, *cache, lens, workspace=workspace, **how)
    n = tv.cache_attention_workspace_bytes(*q.shape[:3], cache[0].shape[2], q.shape[3], cache[0].shape[1])
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    out = fn(q, *cache, lens, workspace=ws, **how)
    assert tv.read_status(ws) == 0
    return out


def _check(kind, q, cache, lens, out, seqs=None, **how):
    seqs = list(range(q.shape[0])) if seqs is None else seqs
    q, lens, cache = q[seqs], lens[seqs], tuple(t[seqs] for t in cache)
    k, v = _values(cache)
    ls = lens.cpu().numpy()
    how = {x: y for x, y in how.items() if x not in ("workspace", "out", "stream")}
    if how.get("slopes") is not None:
        how["slopes"] = _f(how["slopes"])
    want = oc.masked_attention(_f(q), k, v, ls, **how)
    got = _f(out)[seqs]
    assert np.isfinite(got).all()
    D = q.shape[-1]
    for b, L in enumerate(ls):
        if L == 0:
            assert not got[b].any()
            continue
        kk, vv = np.nan_to_num(np.abs(k[b, :L])), np.nan_to_num(np.abs(v[b, :L]), posinf=0)
        V = vv.max()
        G = q.shape[2] // kk.shape[1]
        scale = how.get("scale") or D ** -0.5
        A = max(float((np.abs(_f(q)[b, :, h]) @ kk[:, h // G].T).max()) for h in range(q.shape[2])) * scale
        if how.get("slopes") is not None:
            A += float(np.abs(how["slopes"]).max()) * L
        score = 2.0 ** -18 * A + 2 * 2.0 ** -22 * how.get("softcap", 0.0)
        weight = 2 * 2.0 ** -8 if kind == "masked" else 2.0 ** -11 + 2.0 ** -20 * int(L)
        tol = 2.0 ** -8 * np.abs(want[b]) + (weight + 2 * score) * V * (1 + 2.0 ** -8)
        err = np.abs(got[b] - want[b])
        assert (err <= tol).all(), (kind, b, L, float(err.max()), float((err - tol).max()))


# kv8_keys: the 8-bit cache with unused batch slots added, so that the call goes
# to the form of the kernel for many tiles (head dim 128, up to 32 query rows).
KINDS = ["kv8", "kv8_keys", "masked"]


def _skip_unless_it_applies(kind, D, rows):
    if kind == "kv8_keys" and (D != 128 or rows > 32):
        pytest.skip("the form for many tiles is for head dim 128 and up to 32 query rows")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B,n,Hq,Hkv,D,Lmax", [
    (1, 1, 1, 1, 128, 1),         # one row, one head
    (3, 1, 8, 2, 64, 40),         # single new tokens
    (1, 5, 32, 8, 128, 700),      # Llama grouping, one sequence over many CTAs
    (2, 3, 4, 4, 256, 301),       # wide heads, no grouping
    (5, 8, 16, 2, 128, 333),      # 64 query rows per KV head: one full group
    (2, 9, 16, 2, 128, 290),      # 72 rows: two groups
    (2, 7, 12, 2, 256, 150),      # 42 rows at 256 dims: two groups
    (40, 2, 4, 2, 64, 129),       # more tiles than one CTA's share of each
])
def test_chain_matches_oracle(kind, B, n, Hq, Hkv, D, Lmax):
    _skip_unless_it_applies(kind, D, n * Hq // Hkv)
    q, cache, lens = _inputs(kind, B + Lmax, B, n, Hq, Hkv, D, Lmax)
    _check(kind, q, cache, lens, _call(kind, q, cache, lens))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("how", [
    {"softcap": 5.0}, {"window": 1}, {"window": 37}, {"window": 1000, "softcap": 30.0, "scale": 0.2},
    {"slopes": True}, {"slopes": True, "window": 64, "softcap": 20.0},
    {"parent": TREE26}, {"parent": TREE26, "window": 3}, {"parent": TREE26, "slopes": True, "softcap": 10.0},
], ids=str)
def test_options_match_oracle(kind, D, how):
    n = 26 if "parent" in how else 4
    how = dict(how)
    if kind == "kv8_keys" and n == 26:
        how["parent"], n = TREE26[:16], 16
    _skip_unless_it_applies(kind, D, 2 * n)
    if how.get("slopes"):
        how["slopes"] = torch.tensor([0.5, 0.25, 0.1, 0.01], device=DEV)
    q, cache, lens = _inputs(kind, D + n, 3, n, 4, 2, D, 310, lens=[310, n, 129])
    _check(kind, q, cache, lens, _call(kind, q, cache, lens, **how), **how)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("cap", [1e-3, 0.5, 1000.0])
def test_narrow_and_wide_caps(kind, cap):
    """A cap far below the scores leaves their signs, one far above the scores themselves."""
    q, cache, lens = _inputs(kind, 21, 2, 3, 4, 2, 128, 290, lens=[290, 100])
    _check(kind, q, cache, lens, _call(kind, q, cache, lens, softcap=cap), softcap=cap)


@pytest.mark.parametrize("kind", KINDS)
def test_lengths_around_the_blocks(kind):
    """Lengths on, before and after the edges of 32, 64 and 128 rows, and unused slots."""
    lens = [3, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 0, 258, 0]
    q, cache, lens = _inputs(kind, 11, len(lens), 3, 4, 2, 128, 258, lens=lens)
    _check(kind, q, cache, lens, _call(kind, q, cache, lens))


@pytest.mark.parametrize("kind", ["kv8", "masked"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("how", [{}, {"window": 2500}], ids=str)
def test_long_ragged_batch(kind, D, how):
    """Many blocks that every position sees between those with masks, several tiles per CTA."""
    import target_model_verify_gb300 as tv
    lens = [6000, 40, 5111, 3, 2600, 1, 0, 4097] * 4
    q, cache, lens = _inputs(kind, 22, len(lens), 1, 16, 8, D, 6000, lens=lens)      # 256 tiles
    ws = torch.empty(tv.cache_attention_workspace_bytes(len(lens), 1, 16, 8, D, 6000), dtype=torch.uint8,
                     device=DEV)
    out = _call(kind, q, cache, lens, workspace=ws, **how)
    assert tv.read_status(ws) == 0
    _check(kind, q, cache, lens, out, seqs=[0, 2, 3, 15, 28, 30, 31], **how)


@pytest.mark.parametrize("kind", ["kv8", "masked"])
@pytest.mark.parametrize("n,Hq,Hkv,D,L", [
    (2, 4, 1, 128, 20000),        # one KV head: a tile shared by more CTAs than a warp has lanes
    (2, 4, 2, 256, 9001),
    (40, 1, 1, 64, 5000),         # 64 lanes of query rows
    (9, 16, 2, 128, 4001),        # 72 query rows
    (3, 8, 8, 128, 33001),        # the form for many blocks
])
def test_one_sequence_over_every_cta(kind, n, Hq, Hkv, D, L):
    q, cache, lens = _inputs(kind, L, 1, n, Hq, Hkv, D, L, lens=[L])
    _check(kind, q, cache, lens, _call(kind, q, cache, lens))


@pytest.mark.parametrize("kind", ["kv8", "masked"])
def test_many_kv_heads(kind):
    """More KV heads than can have CTAs side by side."""
    q, cache, lens = _inputs(kind, 23, 2, 2, 200, 100, 64, 300, lens=[300, 131])
    _check(kind, q, cache, lens, _call(kind, q, cache, lens))


def test_many_tiles_in_a_graph():
    """The form for many tiles, captured and replayed on new lengths and queries; twice alike."""
    import target_model_verify_gb300 as tv
    B = 33
    q, cache, lens = _inputs("kv8", 24, B, 4, 32, 8, 128, 333)
    ws = torch.empty(tv.cache_attention_workspace_bytes(B, 4, 32, 8, 128, 333), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = tv.verify_attention_kv8(q, *cache, lens, workspace=ws)
    for step in range(2):
        lens.copy_((lens + 97 * step) % 330 + 4)
        q.copy_(q.flip(0))
        graph.replay()
        first = out.clone()
        graph.replay()
        assert tv.read_status(ws) == 0
        assert torch.equal(out, first)
        assert torch.equal(out, tv.verify_attention_kv8(q, *cache, lens))
        _check("kv8", q, cache, lens, out, seqs=[0, 7, 32])


@pytest.mark.parametrize("kind", ["kv8", "masked"])
def test_deepest_tree(kind):
    """128 nodes: a chain of 64 and leaves hung on it, 4 query heads per KV head (512 rows)."""
    parent = [-1] + list(range(63)) + [5 * i % 64 for i in range(64)]
    q, cache, lens = _inputs(kind, 12, 2, 128, 4, 1, 64, 200, lens=[200, 128])
    _check(kind, q, cache, lens, _call(kind, q, cache, lens, parent=parent, window=50), parent=parent,
           window=50)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_unseen_rows_never_reach_the_output(kind, D):
    """NaN (and infinities) in rows past the length, in later positions' rows, in other branches
    and before the window change nothing; in a visible row they do, for the rows that see it."""
    _skip_unless_it_applies(kind, D, 8)
    parent = (-1, 0, 0, 1)
    q, cache, lens = _inputs(kind, 13, 2, 4, 4, 2, D, 200, lens=[150, 190])
    base = _call(kind, q, cache, lens, parent=parent, window=90)
    bad = float("inf") if kind == "masked" else float("nan")
    k, v = cache[0].float(), cache[1].float()
    for t in (k, v):
        t[0, 150:] = float("nan")
        t[1, 190:] = bad
        t[0, :150 - 4 - 90 + 1] = bad           # out of every position's window
        t[1, 187 + 1] = bad                     # node 2: seen by itself only
    hurt = (k.to(cache[0].dtype), v.to(cache[1].dtype)) + cache[2:]
    out = _call(kind, q, hurt, lens, parent=parent, window=90)
    assert torch.equal(out[0], base[0])
    assert torch.equal(out[1, [0, 1, 3]], base[1, [0, 1, 3]])
    assert out[1, 2].isnan().all()


@pytest.mark.parametrize("kind", KINDS)
def test_value_nan_reaches_who_sees_it(kind):
    """A NaN in one value element of a late row reaches that dim of the rows that see it only."""
    q, cache, lens = _inputs(kind, 14, 1, 4, 4, 2, 128, 300, lens=[300])
    base = _call(kind, q, cache, lens)
    v = cache[1].float()
    v[0, 298, 1, 77] = float("nan")             # new position 2, KV head 1
    v[0, 100, 0, 5] = float("nan")              # seen by all, KV head 0
    out = _call(kind, q, (cache[0], v.to(cache[1].dtype)) + cache[2:], lens)
    want = torch.zeros_like(out, dtype=torch.bool)
    want[0, 2:, 2:, 77] = True
    want[0, :, :2, 5] = True
    assert torch.equal(out.isnan(), want)
    assert torch.equal(out[~want], base[~want])


@pytest.mark.parametrize("kind", KINDS)
def test_bad_lengths_set_the_status(kind):
    import target_model_verify_gb300 as tv
    q, cache, lens = _inputs(kind, 15, 5, 5, 8, 2, 128, 100, lens=[50, 101, 4, -3, 100])
    ws = torch.empty(tv.cache_attention_workspace_bytes(5, 5, 8, 2, 128, 100), dtype=torch.uint8, device=DEV)
    out = torch.full((5, 5, 8, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    assert _call(kind, q, cache, lens, out=out, workspace=ws) is out
    assert tv.read_status(ws) == tv._b.SPECDEC_ERR_INVALID_ARG
    assert not out[1:4].any()
    _check(kind, q, cache, lens, out, seqs=[0, 4])
    lens[1:4] = 0
    _call(kind, q, cache, lens, out=out, workspace=ws)
    assert tv.read_status(ws) == 0


def test_block_scales_of_every_size():
    """Value scales over the whole range: blocks of zeros, of tiny and of huge values side by side."""
    q, cache, lens = _inputs("kv8", 16, 2, 3, 4, 2, 128, 256, lens=[256, 200])
    e = torch.tensor([-40, 20, -6, -40, 0, -20, 3, -6], device=DEV)
    vs = torch.ldexp(torch.ones(8, device=DEV), e).expand(2, 2, 8).contiguous()
    v = cache[1].float()
    v[:, :32] = 0
    cache = (cache[0], v.to(torch.float8_e4m3fn), cache[2], vs)
    _check("kv8", q, cache, lens, _call("kv8", q, cache, lens))


def test_queries_of_every_size():
    """Query rows from 2^-60 to 2^40 (scores of the largest stay finite), zeros among them."""
    q, cache, lens = _inputs("kv8", 17, 1, 5, 4, 2, 64, 100, lens=[100])
    f = torch.ldexp(torch.ones(5, device=DEV), torch.tensor([-60, -20, 0, 3, 40], device=DEV))
    q = (q.float() * f[None, :, None, None]).to(torch.bfloat16)
    q[:, :, 1] = 0
    out = _call("kv8", q, cache, lens)
    _check("kv8", q[:, :4].contiguous(), cache, lens - 1, _call("kv8", q[:, :4].contiguous(), cache, lens - 1))
    # a score gap of 2^30 or more: the row is its best key's value
    k, v = _values(cache)
    for h in (0, 2, 3):
        best = int(np.argmax(k[0, :, h // 2] @ _f(q)[0, 4, h]))
        np.testing.assert_allclose(_f(out)[0, 4, h], v[0, best, h // 2], rtol=2.0 ** -8, atol=0)


@pytest.mark.parametrize("kind", ["kv8", "masked"])
def test_streams_graphs_and_repeats(kind):
    """A fused projection's slice of queries; another stream; a captured call replayed on new
    lengths; equal results every time."""
    import target_model_verify_gb300 as tv
    q0, cache, lens = _inputs(kind, 18, 3, 4, 8, 2, 128, 400, lens=[400, 77, 250])
    fused = torch.randn(3, 4, 12, 128, device=DEV).to(torch.bfloat16)
    fused[:, :, :8] = q0
    q = fused[:, :, :8]
    base = _call(kind, q0, cache, lens)
    assert torch.equal(_call(kind, q, cache, lens), base)
    _check(kind, q0, cache, lens, base)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = _call(kind, q, cache, lens, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, base)
    ws = torch.empty(tv.cache_attention_workspace_bytes(3, 4, 8, 2, 128, 400), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = _call(kind, q, cache, lens, workspace=ws, parent=(-1, 0, 0, 2))
    for new in ([400, 77, 250], [5, 0, 399]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, _call(kind, q, cache, lens, parent=(-1, 0, 0, 2)))
        _check(kind, q0, cache, lens, out, parent=(-1, 0, 0, 2))


def test_long_cache_past_32_bits():
    """A cache of more than 2^32 elements per tensor: the last sequence's rows."""
    import target_model_verify_gb300 as tv
    B, Lmax, H, D = 33, 131072, 8, 128
    k, v, ks, vs = tv.alloc_kv8_cache(B, Lmax, H, D)
    for t in (k, v):
        t.view(torch.uint8).fill_(0x7f)          # NaN everywhere but in the rows used
    ks.fill_(1.0)
    vs.fill_(1.0)
    g = torch.Generator(device=DEV).manual_seed(19)
    new = [torch.randn(B, 5, H, D, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2)]
    start = torch.full((B,), -5, dtype=torch.int32, device=DEV)
    start[0], start[B - 1] = 0, 0
    counts = torch.zeros(B, dtype=torch.int32, device=DEV)
    counts[0] = counts[B - 1] = 5
    tv.append_kv8(*new, k, v, ks, vs, start, counts)
    lens = counts.clone()
    q = torch.randn(B, 5, 8, D, generator=g, device=DEV).to(torch.bfloat16)
    out = tv.verify_attention_kv8(q, k, v, ks, vs, lens)
    pick = [0, B - 1]
    cut = lambda t: t[pick, :64].contiguous() if t.dim() == 4 else t[pick, :, :2].contiguous()  # noqa: E731
    _check("kv8", q[pick], (cut(k), cut(v), ks[pick][:, :, :2], vs[pick][:, :, :2]), lens[pick], out[pick])
    assert not out[1:B - 1].any()


def test_verify_layer_step():
    """The operators as a layer uses them: a prompt appended, a chain step, a rejection, a tree step,
    the accepted path appended again, and a last step on it; each step against the oracle on the
    cache's own values, and the last against a cache that never held the tree."""
    import target_model_verify_gb300 as tv
    g = torch.Generator(device=DEV).manual_seed(20)
    B, Hq, Hkv, D, Lmax = 3, 8, 2, 128, 160
    rnd = lambda n, H: torch.randn(B, n, H, D, generator=g, device=DEV).to(torch.bfloat16)  # noqa: E731
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    cache = tv.alloc_kv8_cache(B, Lmax, Hkv, D)
    prompt = ints([100, 1, 31])
    tv.append_kv8(rnd(100, Hkv), rnd(100, Hkv), *cache, ints([0, 0, 0]), counts=prompt)
    # a chain of 5; the first, all and three of its positions stay
    q, k, v = rnd(5, Hq), rnd(5, Hkv), rnd(5, Hkv)
    tv.append_kv8(k, v, *cache, prompt)
    _check("kv8", q, cache, prompt + 5, tv.verify_attention_kv8(q, *cache, prompt + 5))
    at = prompt + ints([1, 5, 3])
    # a tree of 26 on top
    q, k, v = rnd(26, Hq), rnd(26, Hkv), rnd(26, Hkv)
    twin = tuple(t.clone() for t in cache)
    tv.append_kv8(k, v, *cache, at)
    out = tv.verify_attention_kv8(q, *cache, at + 26, parent=TREE26)
    _check("kv8", q, cache, at + 26, out, parent=TREE26)
    # the accepted path: the root's row stays, out_nodes' rows follow it
    nodes = torch.full((B, 26), -1, dtype=torch.int32, device=DEV)
    nodes[0, :3], nodes[2, :1] = ints([1, 5, 12]), ints([4])
    n_acc = ints([3, 0, 1])
    tv.append_kv8(k, v, *cache, at + 1, counts=n_acc, rows=nodes)
    at = at + 1 + n_acc
    q = rnd(1, Hq)
    k1, v1 = rnd(1, Hkv), rnd(1, Hkv)
    tv.append_kv8(k1, v1, *cache, at)
    out = tv.verify_attention_kv8(q, *cache, at + 1)
    _check("kv8", q, cache, at + 1, out)
    # a cache that never held the rejected nodes: scales differ by what those had, codes by a step
    order = torch.cat([torch.zeros(B, 1, dtype=torch.int32, device=DEV), nodes[:, :25]], 1)
    tv.append_kv8(k, v, *twin, at - 1 - n_acc, counts=n_acc + 1, rows=order)
    tv.append_kv8(k1, v1, *twin, at)
    for b, L in enumerate((at + 1).tolist()):
        for x in (0, 1):
            a = oc.dequantise(_f(cache[x]), _f(cache[2 + x]))[b, :L]
            w = oc.dequantise(_f(twin[x]), _f(twin[2 + x]))[b, :L]
            # each side is within half a step (2^-4, or 2^-10 of the scale) of the value, once or
            # twice rounded; the rejected nodes raise a scale by at most their own magnitude
            step = _f(cache[2 + x])[b, :, :-(-L // 32)].max()
            assert (np.abs(a - w) <= 4 * 2.0 ** -4 * np.abs(w) + 4 * 2.0 ** -10 * step).all()


@pytest.mark.parametrize("kind,B,n,Hq,Hkv,D,Lmax,lens", [
    ("kv8", 3, 5, 32, 8, 128, 300, [300, 0, 129]),        # fewer tiles than CTAs, an unused slot
    ("kv8", 40, 3, 32, 8, 128, 200, None),                # the form for many tiles
    ("kv8", 1, 26, 32, 8, 64, 5000, [5000]),              # 128 lanes, one sequence over every CTA
    ("masked", 2, 40, 16, 2, 256, 150, [150, 40]),        # several row groups
    ("masked", 5, 2, 200, 100, 64, 90, None),             # more heads than CTAs side by side
])
def test_margins_are_left(kind, B, n, Hq, Hkv, D, Lmax, lens):
    """Workspace and output lie between margins of 4 KB; a call writes neither."""
    import target_model_verify_gb300 as tv
    q, cache, lens = _inputs(kind, 30, B, n, Hq, Hkv, D, Lmax, lens=lens)
    sizes = {"workspace": tv.cache_attention_workspace_bytes(B, n, Hq, Hkv, D, Lmax), "out": q.numel() * 2}
    if kind == "masked":
        sizes["workspace"] = tv._b.specdec_verify_attention_masked_workspace_size(B, n, Hq, Hkv, D, Lmax)
    whole = {k: torch.full((v + 8192,), 0xA5, dtype=torch.uint8, device=DEV) for k, v in sizes.items()}
    inner = {k: whole[k][4096:4096 + v] for k, v in sizes.items()}
    inner["out"] = inner["out"].view(torch.bfloat16).view(q.shape)
    out = _call(kind, q, cache, lens, **inner)
    for k, v in sizes.items():
        assert (whole[k][:4096] == 0xA5).all() and (whole[k][4096 + v:] == 0xA5).all(), k
    assert tv.read_status(inner["workspace"]) == 0
    _check(kind, q, cache, lens, out)


def test_refusals():
    import target_model_verify_gb300 as tv
    q, cache, lens = _inputs("kv8", 21, 2, 3, 4, 2, 128, 64)
    k, v, ks, vs = cache
    b16 = k.to(torch.bfloat16)
    for call, err in (
            (lambda: tv.verify_attention_kv8(q.float(), *cache, lens), TypeError),
            (lambda: tv.verify_attention_kv8(q, b16, b16, ks, vs, lens), TypeError),
            (lambda: tv.verify_attention_masked(q, k, v, lens), TypeError),
            (lambda: tv.verify_attention_kv8(q, k, v, ks[:, :, :1].contiguous(), vs, lens), ValueError),
            (lambda: tv.verify_attention_kv8(q, *cache, lens.long()), TypeError),
            (lambda: tv.verify_attention_kv8(q, *cache, lens[:1]), ValueError),
            (lambda: tv.verify_attention_kv8(q[:1], *cache, lens), ValueError),
            (lambda: tv.verify_attention_kv8(q.transpose(1, 2), *cache, lens), ValueError),
            (lambda: tv.verify_attention_kv8(q, *cache, lens, parent=(-1, 0)), ValueError),
            (lambda: tv.verify_attention_kv8(q, *cache, lens, parent=(-1, 0, 2)), tv.SpecdecError),
            (lambda: tv.verify_attention_kv8(q, *cache, lens, window=-1), tv.SpecdecError),
            (lambda: tv.verify_attention_kv8(q, *cache, lens, softcap=-1.0), tv.SpecdecError),
            (lambda: tv.verify_attention_kv8(q, *cache, lens, slopes=torch.ones(2, device=DEV)), ValueError),
            (lambda: tv.verify_attention_kv8(q, *cache, lens, workspace=torch.empty(64, dtype=torch.uint8,
                                                                                    device=DEV)),
             tv.SpecdecError),
            (lambda: tv.verify_attention_kv8(q, *cache, lens.cpu()), TypeError),
            (lambda: tv.append_kv8(q, q, *cache, lens), ValueError),
            (lambda: tv.append_kv8(b16.float(), b16, *cache, lens), TypeError),
            (lambda: tv.append_kv8(b16, b16, *cache, lens.float()), TypeError),
            (lambda: tv.append_kv8(b16.transpose(1, 2), b16.transpose(1, 2), *cache, lens), ValueError),
            (lambda: tv.append_kv8(b16, b16, *cache, lens, rows=lens), ValueError)):
        with pytest.raises(err):
            call()
