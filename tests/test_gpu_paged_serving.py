"""The paged cache's operators together, as a serving loop uses them: prompts, their pages, steps of a
drafter's token, of a chain and of a tree with rejections, requests that end and others in their place.
Every attention is compared with the fp64 oracle over the whole history kept on the host."""
import numpy as np
import pytest
import torch

from oracle import cache as oc
from oracle import prompt as opr
from tests.test_gpu_cache_attention import TREE26

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _f(t):
    return t.detach().float().cpu().double().numpy()


def _i(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _close(got, want, V):
    # the output's rounding, the weights' (2^-8 each, in the product alone or with the sum), the scores' within it
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 3 * 2.0 ** -8 * V).all(), float(np.abs(got - want).max())


@pytest.mark.parametrize("D,page,how", [(128, 16, {}), (64, 32, {"window": 150}), (256, 64, {"softcap": 30.0})], ids=str)
def test_serving_loop(D, page, how):
    import target_model_verify_gb300 as tv
    Hq, Hkv, B, max_pages, n_pages = 4, 2, 4, 512 // page, 4 * 400 // page
    g = torch.Generator(device=DEV).manual_seed(D)
    rng = np.random.default_rng(D)
    pool = tv.alloc_paged_cache(n_pages, page, Hkv, D, device=DEV)
    for t in pool:
        t.fill_(float("nan"))                          # nothing but what was written may be read
    tables = tv.alloc_page_tables(B, max_pages, n_pages, device=DEV)
    ws = torch.empty(1 << 26, dtype=torch.uint8, device=DEV)
    history = [(np.zeros((0, Hkv, D)), np.zeros((0, Hkv, D))) for _ in range(B)]
    lens = [0] * B

    def new(*shape):
        qkv = torch.randn(*shape, Hq + 2 * Hkv, D, generator=g, device=DEV).to(torch.bfloat16)
        return qkv.split([Hq, Hkv, Hkv], dim=-2)

    def ok():
        assert tv.read_status(ws) == 0

    def admit(slots_of, count):
        """Prompts of `count` tokens into empty slots of the batch, packed."""
        cu = [0]
        for b in range(B):
            cu.append(cu[-1] + (count[slots_of.index(b)] if b in slots_of else 0))
        q, k, v = new(cu[-1])
        out = tv.prompt_attention(q, k, v, _i(cu), workspace=ws, **how)
        ok()
        want, _ = opr.attention(_f(q), _f(k), _f(v), cu, **how)
        _close(_f(out), want, np.abs(_f(v)).max())
        slots = tv.plan_pages(*tables, _i([0 if b in slots_of else lens[b] for b in range(B)]),
                              _i([cu[b + 1] - cu[b] for b in range(B)]), page, n=cu[-1], cu_rows=_i(cu), workspace=ws)
        ok()
        tv.append_paged(k, v, *pool, slots, workspace=ws)
        ok()
        for b in slots_of:
            history[b] = (_f(k[cu[b]:cu[b + 1]]), _f(v[cu[b]:cu[b + 1]]))
            lens[b] = cu[b + 1] - cu[b]

    def step(n, parent=None):
        """One step of n new positions for every live sequence; some of them are kept."""
        live = [n if lens[b] else 0 for b in range(B)]
        q, k, v = new(B, n)
        k, v = k.contiguous(), v.contiguous()
        start = _i(lens)
        slots = tv.plan_pages(*tables, start, _i(live), page, n=n, workspace=ws)
        ok()
        tv.append_paged(k, v, *pool, slots, workspace=ws)
        ok()
        total = [lens[b] + live[b] for b in range(B)]
        out = tv.verify_attention_paged(q, *pool, tables[0], _i(total), parent=parent, workspace=ws, **how)
        ok()
        for b in range(B):
            if not live[b]:
                assert not out[b].any()
                continue
            kk, vv = (np.concatenate([history[b][x], _f(t[b])])[None] for x, t in ((0, k), (1, v)))
            want = oc.masked_attention(_f(q[b:b + 1]), kk, vv, [total[b]], parent=parent, **how)
            _close(_f(out[b:b + 1]), want, np.abs(vv).max())
        if parent is None:
            kept = [int(rng.integers(1, n + 1)) if live[b] else 0 for b in range(B)]
            tv.plan_pages(*tables, start, _i(kept), page, workspace=ws)
            ok()
            rows = [list(range(c)) for c in kept]
        else:
            # a path from the root: the accepted nodes replace the tree behind the root's row
            rows = []
            for b in range(B):
                path = [0]
                while live[b] and rng.random() < 0.8:
                    kids = [c for c in range(n) if parent[c] == path[-1]]
                    if not kids:
                        break
                    path.append(int(rng.choice(kids)))
                rows.append(path if live[b] else [])
            kept = [len(r) for r in rows]
            after = [max(c - 1, 0) for c in kept]
            nodes = np.full((B, n), -1)
            for b in range(B):
                nodes[b, :after[b]] = rows[b][1:]
            slots = tv.plan_pages(*tables, _i([lens[b] + (1 if live[b] else 0) for b in range(B)]), _i(after), page, n=n,
                                  workspace=ws)
            ok()
            tv.append_paged(k, v, *pool, slots, rows=_i(nodes.tolist()), workspace=ws)
            ok()
        for b in range(B):
            if live[b]:
                history[b] = tuple(np.concatenate([history[b][x], _f(t[b])[rows[b]]]) for x, t in ((0, k), (1, v)))
                lens[b] += kept[b]
        held = [-(-x // page) for x in lens]
        assert tables[1].tolist() == held and tables[3].item() == n_pages - sum(held)

    admit([0, 2], [200, 37])
    for n in (1, 5, 1):
        step(n)
    admit([1, 3], [3 * page + 1, 1])
    step(26, parent=TREE26)
    step(1)
    step(9)
    lens[0] = 0                                        # a request ends
    tv.plan_pages(*tables, _i(lens), _i([0] * B), page, workspace=ws)
    ok()
    step(5)
    admit([0], [300])                                  # another in its place, in pages given back
    step(12, parent=TREE26[:12])
    step(2)


def test_outputs_and_workspaces_keep_to_their_bounds():
    """Bytes before and behind every output, and behind a workspace of the stated size, stay as they were."""
    import target_model_verify_gb300 as tv
    g = torch.Generator(device=DEV).manual_seed(3)

    def guarded(nbytes):
        big = torch.full((nbytes + 2048,), 0x5a, dtype=torch.uint8, device=DEV)
        return big, big[1024:1024 + nbytes]

    def intact(big, nbytes):
        assert (big[:1024] == 0x5a).all() and (big[1024 + nbytes:] == 0x5a).all()

    for D, n, Hq, Hkv in ((64, 1, 8, 2), (128, 9, 8, 2), (256, 2, 6, 2)):
        B, page, lens = 3, 16, [70, 33, 16]
        pages = [torch.randn(12, page, Hkv, D, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2)]
        table = _i([[0, 1, 2, 3, 4], [5, 6, 7, -1, -1], [8, -1, -1, -1, -1]])
        q = torch.randn(B, n, Hq, D, generator=g, device=DEV).to(torch.bfloat16)
        size = tv.paged_attention_workspace_bytes(B, n, Hq, Hkv, D, 12, page, 5)
        (big_ws, ws), (big_out, out) = guarded(size), guarded(q.numel() * 2)
        tv.verify_attention_paged(q, *pages, table, _i(lens), out=out.view(torch.bfloat16).view(q.shape), workspace=ws)
        assert tv.read_status(ws) == 0
        intact(big_ws, size), intact(big_out, q.numel() * 2)
        T, cu = 333, [0, 100, 333]
        q, k, v = (torch.randn(T, h, D, generator=g, device=DEV).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
        size = tv.prompt_attention_workspace_bytes(2, T, Hq, Hkv, D)
        (big_ws, ws), (big_out, out) = guarded(size), guarded(q.numel() * 2)
        tv.prompt_attention(q, k, v, _i(cu), out=out.view(torch.bfloat16).view(q.shape), workspace=ws)
        assert tv.read_status(ws) == 0
        intact(big_ws, size), intact(big_out, q.numel() * 2)
    tables = [guarded(4 * x) for x in (3 * 7, 3, 30, 1)]
    views = [t.view(torch.int32) for _, t in tables]
    for view, fresh in zip(views, tv.alloc_page_tables(3, 7, 30, device=DEV)):
        view.copy_(fresh.flatten())
    big_ws, ws = guarded(256)
    big_map, smap = guarded(4 * 3 * 5)
    for counts in ([5, 5, 5], [1, 0, 3]):
        tv.plan_pages(views[0].view(3, 7), *views[1:], _i([100, 0, 31]), _i(counts), 16,
                      slots=smap.view(torch.int32).view(3, 5), workspace=ws)
        assert tv.read_status(ws) == 0
    for (big, t), size in zip(tables, (84, 12, 120, 4)):
        intact(big, size)
    intact(big_ws, 256), intact(big_map, 60)


def test_pool_beyond_32_bits():
    """Rows whose elements lie past 2^32 bytes and 2^31 elements of their tensor."""
    import target_model_verify_gb300 as tv
    Hkv, D, page = 8, 128, 256
    n_pages = (1 << 31) // (page * Hkv * D) + 40            # 4.4 GB each
    pool = tv.alloc_paged_cache(n_pages, page, Hkv, D, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(4)
    for n in (1, 5):                                        # 4 rows, and 20: both forms
        ids = [n_pages - 1, 0, n_pages - 7, n_pages - 30]
        L = 4 * page - 9
        q = torch.randn(1, n, 32, D, generator=g, device=DEV).to(torch.bfloat16)
        new = [torch.randn(L, Hkv, D, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2)]
        slots = _i([ids[j // page] * page + j % page for j in range(L)])
        tv.append_paged(*new, *pool, slots)
        for t, x in zip(pool, new):
            assert torch.equal(torch.cat([t[p] for p in ids])[:L], x)
        out = tv.verify_attention_paged(q, *pool, _i([ids]), _i([L]))
        want = oc.masked_attention(_f(q), _f(new[0])[None], _f(new[1])[None], [L])
        _close(_f(out), want, np.abs(_f(new[1])).max())


def test_prompt_strides_beyond_32_bits():
    """Tokens 2^26 elements apart: the last ones' rows lie past 2^32 bytes and 2^31 elements."""
    import target_model_verify_gb300 as tv
    T, stride, D = 50, 1 << 26, 128
    base = torch.empty(T * stride, dtype=torch.bfloat16, device=DEV)
    rows = base.view(T, stride)[:, :12 * D].view(T, 12, D)
    rows.copy_(torch.randn(T, 12, D, device=DEV))
    q, k, v = rows.split([8, 2, 2], dim=1)
    v[3, 0, 5] = float("inf")                               # and where values are looked up again
    out = tv.prompt_attention(q, k, v, _i([0, 20, T]))
    assert (out[3:20, :4, 5] == float("inf")).all()
    want, _ = opr.attention(_f(q), _f(k), np.nan_to_num(_f(v), posinf=0), [0, 20, T])
    got = _f(out)
    got[3:20, :4, 5] = want[3:20, :4, 5] = 0
    _close(got, want, 5.0)
