"""What the cache operators' calls promise at their edges, on the GPU: tables that end early, options at
the ends of their ranges, workspaces, many query heads per KV head."""
import numpy as np
import pytest
import torch

from oracle import cache as oc
from tests.test_gpu_cache_attention import _call, _check, _inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _f(t):
    return t.detach().float().cpu().double().numpy()


def _i(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("n,counts", [(5, [5, 0, 2]), (40, [0, 40, 33]), (26, [3, 26, 0])])
def test_rows_table_may_end_with_the_last_count(n, counts):
    """The C call with a table that ends behind the last entry the counts name: what is not named is not
    read (the memory behind it holds entries that would not pass)."""
    import target_model_verify_gb300 as tv
    b = tv._b
    g = torch.Generator(device=DEV).manual_seed(1)
    B, H, D, Lmax = 3, 2, 64, 160
    new = [torch.randn(B, n, H, D, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2)]
    cache = tv.alloc_kv8_cache(B, Lmax, H, D, device=DEV)
    for t in cache[:2]:
        t.view(torch.uint8).fill_(0x30)
    for t in cache[2:]:
        t.fill_(2.0 ** -8)
    start = [0, 31, 100]
    table = np.full((B, n), -1)
    for s, c in enumerate(counts):
        table[s, :c] = np.arange(c)[::-1]
    last = max(s for s in range(B) if counts[s])
    used = last * n + counts[last]
    whole = torch.full((B * n,), 1 << 30, dtype=torch.int32, device=DEV)       # in one piece: nothing is out of bounds
    whole[:used] = _i(table.reshape(-1)[:used].tolist())
    for s, c in enumerate(counts):
        whole[s * n + c:(s + 1) * n] = -(1 << 30)
    want = [oc.append(_f(new[x]), _f(cache[x]), _f(cache[2 + x]), start, counts, table) for x in (0, 1)]
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    st, ct = _i(start), _i(counts)
    rc = b.specdec_kv8_append(new[0].data_ptr(), H * D, new[1].data_ptr(), H * D, st.data_ptr(), ct.data_ptr(),
                              whole.data_ptr(), B, n, H, D, Lmax, *(t.data_ptr() for t in cache), ws.data_ptr(), 256,
                              torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and tv.read_status(ws) == 0
    for x in (0, 1):
        np.testing.assert_array_equal(_f(cache[2 + x]), want[x][1])
        np.testing.assert_array_equal(_f(cache[x]), want[x][0])


@pytest.mark.parametrize("B,D", [(3, 64), (130, 128)])
@pytest.mark.parametrize("kind", ["kv8", "masked"])
@pytest.mark.parametrize("parent", [None, (-1, 0, 0, 1, 3)], ids=str)
def test_windows_to_the_end_of_32_bits(kind, B, D, parent):
    """A window that no distance reaches is none, whatever its size; one that leaves out the first row
    of the longest sequence alone does that."""
    import target_model_verify_gb300 as tv
    g = torch.Generator(device=DEV).manual_seed(2)
    n, Hq, Hkv, Lmax = 5, 4, 2, 200
    q = torch.randn(B, n, Hq, D, generator=g, device=DEV).to(torch.bfloat16)
    k, v = (torch.randn(B, Lmax, Hkv, D, generator=g, device=DEV) for _ in range(2))
    lens = torch.full((B,), Lmax, dtype=torch.int32, device=DEV)
    lens[1] = 77
    if kind == "masked":
        cache = [k.to(torch.bfloat16), v.to(torch.bfloat16)]
        call = lambda **how: tv.verify_attention_masked(q, *cache, lens, parent=parent, **how)      # noqa: E731
        val = [_f(t[:2]) for t in cache]
    else:
        one = torch.ones(B, Hkv, 7, device=DEV)
        cache = [k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn)]
        call = lambda **how: tv.verify_attention_kv8(q, *cache, one, one, lens, parent=parent, **how)   # noqa: E731
        val = [_f(t[:2]) for t in cache]
    base = call()
    for window in (Lmax, Lmax + 1, 2 ** 31 - 200, 2 ** 31 - 2, 2 ** 31 - 1, 2 ** 31, 2 ** 40):
        assert torch.equal(call(window=window), base), window
    top = Lmax - 1 if parent is None else Lmax - n + 3       # the deepest position's
    got = _f(call(window=top)[:2])
    want = oc.masked_attention(_f(q[:2]), *val, lens[:2].cpu().numpy(), window=top, parent=parent)
    free = oc.masked_attention(_f(q[:2]), *val, lens[:2].cpu().numpy(), parent=parent)
    assert np.abs(want[0, -1] - free[0, -1]).max() > 1e-4 and np.abs(want[1] - free[1]).max() == 0
    # 2^-8 of the output and of the largest value (the weights), twice over for the scores
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 4 * 2.0 ** -8 * np.abs(val[1]).max()).all()


def test_own_workspace_is_of_the_calls_own_size():
    """A call without a workspace takes what its own size function says, and gives it back."""
    import target_model_verify_gb300 as tv
    shape = (4, 5, 32, 8, 128, 300)
    B, n, Hq, Hkv, D, L = shape
    b = tv._b
    sizes = {"kv8": b.specdec_verify_attention_kv8_workspace_size(*shape),
             "masked": b.specdec_verify_attention_masked_workspace_size(*shape)}
    assert sizes["masked"] <= 0.75 * sizes["kv8"]               # else this shape shows nothing
    q = torch.zeros(B, n, Hq, D, dtype=torch.bfloat16, device=DEV)
    out = torch.empty_like(q)
    lens = torch.full((B,), L, dtype=torch.int32, device=DEV)
    k8 = torch.zeros(B, L, Hkv, D, device=DEV).to(torch.float8_e4m3fn)
    one = torch.ones(B, Hkv, -(-L // 32), device=DEV)
    k16 = torch.zeros(B, L, Hkv, D, dtype=torch.bfloat16, device=DEV)
    for kind, call in (("kv8", lambda: tv.verify_attention_kv8(q, k8, k8, one, one, lens, out=out)),
                       ("masked", lambda: tv.verify_attention_masked(q, k16, k16, lens, out=out))):
        call()
        torch.cuda.synchronize()
        held = torch.cuda.memory_allocated()
        torch.cuda.reset_peak_memory_stats()
        call()
        assert torch.cuda.memory_allocated() == held
        took = torch.cuda.max_memory_allocated() - held
        assert sizes[kind] <= took <= sizes[kind] + 512, (kind, took, sizes)


def test_numbers_too_small_for_fp32_are_refused():
    """As fp32 they would be 0, which selects the default scale, or no cap."""
    import target_model_verify_gb300 as tv
    q = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16, device=DEV)
    k8 = torch.zeros(1, 40, 2, 64, device=DEV).to(torch.float8_e4m3fn)
    one = torch.ones(1, 2, 2, device=DEV)
    lens = _i([40])
    for how in ({"scale": 1e-50}, {"softcap": 1e-50}, {"scale": 1e-38}, {"scale": 1e31}, {"scale": float("inf")},
                {"softcap": float("nan")}, {"scale": float("nan")}):
        with pytest.raises(tv.SpecdecError):
            tv.verify_attention_kv8(q, k8, k8, one, one, lens, **how)
        with pytest.raises(tv.SpecdecError):
            tv.verify_attention_masked(q, k8.to(torch.bfloat16), k8.to(torch.bfloat16), lens, **how)


@pytest.mark.parametrize("kind", ["kv8", "kv8_keys", "masked"])
@pytest.mark.parametrize("B,n,Hq,Hkv,D,Lmax,how", [
    (2, 3, 16, 1, 128, 200, {}),                   # 16 query heads per KV head: 48 rows
    (1, 5, 128, 1, 64, 150, {"window": 33}),       # 128: a group of rows per position
    (2, 2, 192, 2, 256, 140, {"softcap": 9.0}),    # 96
    (2, 4, 14, 2, 128, 260, {"window": 100}),      # 7
    (1, 26, 40, 8, 64, 300, {}),                   # 5, 130 rows: two groups of 13 positions
    (2, 6, 8, 2, 128, 300, {}),                    # 24 rows: the most that the form by keys takes
    (2, 3, 16, 2, 128, 300, {"softcap": 9.0}),     # 24
    (2, 25, 2, 2, 128, 300, {}),                   # 25: one more
    (2, 8, 8, 2, 128, 300, {"window": 150}),       # 32
])
def test_query_heads_per_kv_head(kind, B, n, Hq, Hkv, D, Lmax, how):
    q, cache, lens = _inputs(kind, B + Hq, B, n, Hq, Hkv, D, Lmax)
    _check(kind, q, cache, lens, _call(kind, q, cache, lens, **how), **how)


@pytest.mark.parametrize("kind,B,D", [("kv8", 3, 128), ("kv8", 1, 256), ("masked", 2, 256)])
def test_many_kv_heads_in_every_form(kind, B, D):
    """More KV heads than can have CTAs side by side; the first in the form for many tiles."""
    q, cache, lens = _inputs(kind, 31, B, 2, 200, 100, D, 300, lens=[300, 131, 2][:B])
    _check(kind, q, cache, lens, _call(kind, q, cache, lens))


def _layer(seed, B, n, Hq, Hkv, D, Lmax):
    """One layer's step as a program holds it, and the call that runs it: append, then both attentions."""
    import target_model_verify_gb300 as tv
    g = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV).to(torch.bfloat16)     # noqa: E731
    cache = tv.alloc_kv8_cache(B, Lmax, Hkv, D, device=DEV)
    tv.append_kv8(rnd(B, Lmax, Hkv, D), rnd(B, Lmax, Hkv, D), *cache, torch.zeros(B, dtype=torch.int32, device=DEV))
    q, k, v = rnd(B, n, Hq, D), rnd(B, n, Hkv, D), rnd(B, n, Hkv, D)
    kb, vb = rnd(B, Lmax, Hkv, D), rnd(B, Lmax, Hkv, D)
    lens = torch.randint(n + 40, Lmax + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
    start = lens - n

    def step():
        tv.append_kv8(k, v, *cache, start)
        a = tv.verify_attention_kv8(q, *cache, lens)
        tv.append_kv8(v, k, *cache, start)                     # over the same rows: the next call sees these
        b = tv.verify_attention_kv8(q, *cache, lens, softcap=20.0, window=50)
        c = tv.verify_attention_masked(q, kb, vb, lens, window=90)
        tv.append_kv8(k, v, *cache, start)
        return a, b, c
    return step


def test_steps_on_two_streams_and_in_graphs():
    """Steps of two layers, each a chain of calls that begin before the last one ends: run alone, side by
    side on two streams, and captured and replayed side by side, they give the same bits."""
    layers = [_layer(1, 40, 5, 16, 8, 128, 700), _layer(2, 3, 26, 16, 4, 128, 900), _layer(3, 5, 4, 8, 2, 256, 300)]
    layers = [(layers[0], layers[1]), (layers[0], layers[2]), (layers[1], layers[2])]
    for pair in layers:
        alone = []
        for step in pair:
            step()
            torch.cuda.synchronize()
            alone.append([t.clone() for t in step()])
            torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in pair]
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        got = [[], []]
        for _ in range(6):
            for x, (step, s) in enumerate(zip(pair, streams)):
                with torch.cuda.stream(s):
                    got[x].append(step())
        torch.cuda.synchronize()
        graphs, outs = [], []
        for step, s in zip(pair, streams):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                outs.append([step() for _ in range(3)])
            graphs.append(graph)
        for _ in range(4):
            for graph, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    graph.replay()
        torch.cuda.synchronize()
        for x in (0, 1):
            for one in got[x] + outs[x]:
                for a, b in zip(one, alone[x]):
                    assert torch.equal(a, b)


def test_parent_in_every_form_that_verify_tree_takes():
    """Lists, tuples, arrays, tensors and iterators of ints; nothing else."""
    import target_model_verify_gb300 as tv
    q, cache, lens = _inputs("kv8", 40, 2, 5, 4, 2, 64, 90, lens=[90, 40])
    tree = [-1, 0, 0, 1, 3]
    base = _call("kv8", q, cache, lens, parent=tree)
    _check("kv8", q, cache, lens, base, parent=tree)
    for parent in (tuple(tree), np.array(tree), np.array(tree, dtype=np.int32), torch.tensor(tree), iter(tree),
                   (p for p in tree), map(int, tree)):
        assert torch.equal(tv.verify_attention_kv8(q, *cache, lens, parent=parent), base), type(parent)
    for parent in ([-1, 0, 0, 1, 2 ** 40], [-1, 0, 0, 1, 1.5], [-1, 0, 0, 1, None], "abcde", 5, [[-1], [0], [0], [1], [3]]):
        with pytest.raises(TypeError):
            tv.verify_attention_kv8(q, *cache, lens, parent=parent)
    for parent in ([], tree[:4], iter(tree[:2])):
        with pytest.raises(ValueError):
            tv.verify_attention_kv8(q, *cache, lens, parent=parent)


@pytest.mark.parametrize("kind", ["kv8", "masked"])
def test_an_output_from_another_stream_outlives_its_readers(kind):
    """A result of a call on a side stream, read on the current one and dropped there: the side stream
    does not get its memory while the reader still runs."""
    q, cache, lens = _inputs(kind, 41, 3, 4, 8, 2, 128, 150)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = _call(kind, q, cache, lens, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(200_000_000)                     # about 0.1 s
    kept = out.clone()
    at, size = out.data_ptr(), out.numel() * 2
    del out
    with torch.cuda.stream(side):
        held = [torch.empty(size, dtype=torch.uint8, device=DEV) for _ in range(4)]
        for t in held:
            t.fill_(0xFF)
    assert not torch.cuda.current_stream().query(), "the reader was to be running still"
    assert at not in [t.data_ptr() for t in held]
    torch.cuda.synchronize()
    assert torch.equal(kept, _call(kind, q, cache, lens))


@pytest.mark.parametrize("Hq", [8, 32])
def test_a_timeout_outranks_a_bad_length(Hq):
    """What a wait that runs out does to the status word (its code where the word is 0), done by copies on
    another stream while a call of a millisecond or more with one bad length runs: the timeout's code
    stays. (One query row per KV head goes to the form by keys, 104 to the other.)"""
    import target_model_verify_gb300 as tv
    B, n, Hkv, D, L = 32, 1 if Hq == 8 else 26, 8, 128, 1 << 17
    q = torch.zeros(B, n, Hq, D, dtype=torch.bfloat16, device=DEV)
    cache = tv.alloc_kv8_cache(B, L, Hkv, D, device=DEV)
    for t in cache[:2]:
        t.view(torch.uint8).fill_(0x30)
    for t in cache[2:]:
        t.fill_(2.0 ** -6)
    lens = torch.full((B,), L, dtype=torch.int32, device=DEV)
    lens[3] = L + 1
    ws = torch.empty(tv.cache_attention_workspace_bytes(B, n, Hq, Hkv, D, L), dtype=torch.uint8, device=DEV)
    word, out = ws[:4].view(torch.int32), torch.empty_like(q)
    call = lambda: tv.verify_attention_kv8(q, *cache, lens, out=out, workspace=ws)   # noqa: E731
    call()
    assert tv.read_status(ws) == tv._b.SPECDEC_ERR_INVALID_ARG
    seen = torch.zeros(1, dtype=torch.int32).pin_memory()
    timeout = torch.full((1,), tv._b.SPECDEC_ERR_TIMEOUT, dtype=torch.int32).pin_memory()
    side, done = torch.cuda.Stream(), torch.cuda.Event()
    for _ in range(20):
        word.fill_(77)                                   # until the call begins
        torch.cuda.synchronize()
        call()
        done.record()
        with torch.cuda.stream(side):
            for _ in range(1000):
                seen.copy_(word, non_blocking=True)
                side.synchronize()
                if seen.item() != 77:
                    break
            if seen.item() == 0:
                word.copy_(timeout, non_blocking=True)
                side.synchronize()
        if not done.query():                             # the copies came in time
            break
    else:
        pytest.fail("the call never ran long enough")
    assert tv.read_status(ws) == tv._b.SPECDEC_ERR_TIMEOUT
    call()
    assert tv.read_status(ws) == tv._b.SPECDEC_ERR_INVALID_ARG
    lens[3] = L
    call()
    assert tv.read_status(ws) == 0
