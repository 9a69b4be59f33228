"""The paged cache's calls check their arguments on the host before anything reaches a GPU, and
the plain-Python tables that the GPU tests compare with hold what they promise (CPU)."""
import ctypes
import random

import numpy as np
import pytest
import torch

from oracle import paged as op
from target_model_verify_gb300 import _binding as b
from target_model_verify_gb300 import build as libbuild

P, WS, BIG = 4096, 4096 * 256, 1 << 30


@pytest.fixture(scope="module", autouse=True)
def _lib():
    libbuild.build()
    b.lib()


# Fake but aligned addresses: every check below fails before any access.

def _plan(table=P, held=P, free=P, n_free=P, start=P, counts=P, cu=0, B=2, max_pages=8, n_pages=64, page=16, n=5,
          n_slots=10, slots=P, ws=WS, nb=BIG):
    return b.specdec_plan_pages(table, held, free, n_free, start, counts, cu, B, max_pages, n_pages, page, n, n_slots,
                                slots, ws, nb, None)


def test_plan_argument_errors():
    assert b.specdec_plan_pages_workspace_size() == 256
    assert _plan(B=0, n_slots=0, table=0, free=0, ws=0) == b.SPECDEC_OK
    assert _plan(B=0, slots=0, table=0, free=0, ws=0) == b.SPECDEC_OK
    for bad in ({"B": -1}, {"max_pages": 0}, {"n_pages": 0}, {"page": 0}, {"page": 8}, {"page": 48}, {"page": 512},
                {"page": -16}, {"max_pages": (1 << 26) + 1}, {"n_pages": (1 << 26) + 1}, {"n_slots": -1},
                {"n_slots": (1 << 31) - 4}):
        assert _plan(**bad) == b.SPECDEC_ERR_UNSUPPORTED, bad
    for bad in ({"table": 0}, {"held": 0}, {"free": 0}, {"n_free": 0}, {"start": 0}, {"counts": 0}, {"table": P + 2},
                {"held": P + 1}, {"free": P + 3}, {"n_free": P + 2}, {"start": P + 2}, {"counts": P + 1}, {"cu": P + 2},
                {"slots": P + 2}, {"n": 4}, {"n": -1}, {"n_slots": 11}, {"slots": 0, "cu": P}):
        assert _plan(**bad) == b.SPECDEC_ERR_INVALID_ARG, bad
    for bad in ({"ws": 0}, {"ws": WS + 8}, {"nb": 255}):
        assert _plan(**bad) == b.SPECDEC_ERR_WORKSPACE, bad


def _append(k=P, ks=1024, v=P, vs=1024, slots=P, rows=0, B=1, n=5, H=8, D=128, n_pages=4, page=16, kp=P, vp=P, ws=WS,
            nb=BIG):
    return b.specdec_paged_append(k, ks, v, vs, slots, rows, B, n, H, D, n_pages, page, kp, vp, ws, nb, None)


def test_append_argument_errors():
    assert b.specdec_paged_append_workspace_size() == 256
    assert _append(B=0, k=0, ws=0) == b.SPECDEC_OK
    assert _append(n=0, k=0, ws=0) == b.SPECDEC_OK
    for bad in ({"D": 96}, {"n": -1}, {"H": 0}, {"H": (1 << 20) + 1}, {"B": -1}, {"page": 24}, {"n_pages": 0},
                {"n_pages": (1 << 26) + 1}, {"n_pages": 1 << 26, "H": 16}, {"B": 1 << 16, "n": 1 << 15}):
        assert _append(**bad) == b.SPECDEC_ERR_UNSUPPORTED, bad
    for bad in ({"k": 0}, {"v": 0}, {"slots": 0}, {"kp": 0}, {"vp": 0}, {"k": P + 2}, {"vp": P + 8}, {"slots": P + 2},
                {"rows": P + 1}, {"ks": 1016}, {"vs": 1028}, {"ks": -1024}, {"vs": 1 << 31}):
        assert _append(**bad) == b.SPECDEC_ERR_INVALID_ARG, bad
    for bad in ({"ws": 0}, {"ws": WS + 8}, {"nb": 255}):
        assert _append(**bad) == b.SPECDEC_ERR_WORKSPACE, bad


def _attend(q=P, qs=4096, kp=P, vp=P, table=P, lens=P, parent=None, slopes=0, B=1, n=5, Hq=32, H=8, D=128, n_pages=4,
            page=16, max_pages=4, scale=0.0, cap=0.0, window=0, out=P, ws=WS, nb=BIG):
    par = 0 if parent is None else ctypes.addressof((ctypes.c_int32 * len(parent))(*parent))
    return b.specdec_verify_attention_paged(q, qs, kp, vp, table, lens, par, slopes, B, n, Hq, H, D, n_pages, page,
                                            max_pages, scale, cap, window, out, ws, nb, None)


def test_attention_argument_errors():
    size = b.specdec_verify_attention_paged_workspace_size
    need = size(1, 5, 32, 8, 128, 4, 16, 4)
    assert need >= 2 * 152 * 20 * 130 * 4
    assert size(1024, 5, 32, 8, 128, 1 << 20, 16, 1 << 12) == need          # grows with neither B nor the pool
    assert _attend(B=0, q=0, ws=0) == b.SPECDEC_OK
    for bad in ({"D": 96}, {"n": 0}, {"n": 129}, {"Hq": 30}, {"Hq": 4}, {"H": 0}, {"B": -1}, {"page": 1},
                {"page": 512}, {"n_pages": 0}, {"max_pages": 0}, {"n_pages": (1 << 26) + 1},
                {"max_pages": (1 << 26) + 1}, {"n": 65, "Hq": 8}, {"Hq": 129 * 8}, {"B": 1 << 25},
                {"n_pages": 1 << 26, "H": 32}):
        assert _attend(**bad) == b.SPECDEC_ERR_UNSUPPORTED, bad
        shape = dict(B=1, n=5, Hq=32, H=8, D=128, n_pages=4, page=16, max_pages=4)
        shape.update(bad)
        assert size(*shape.values()) == 0, bad
    for bad in ({"q": 0}, {"kp": 0}, {"vp": 0}, {"lens": 0}, {"table": 0}, {"table": P + 2}, {"out": 0}, {"q": P + 8},
                {"out": P + 2}, {"lens": P + 2}, {"slopes": P + 1}, {"qs": 4095}, {"qs": 4088}, {"qs": 4100},
                {"qs": 1 << 31}, {"scale": float("nan")}, {"cap": -1.0}, {"cap": 1001.0}, {"window": -1},
                {"parent": (0, 0, 0, 0, 0)}, {"parent": (-1, 0, 0, 3, 0)}):
        assert _attend(**bad) == b.SPECDEC_ERR_INVALID_ARG, bad
    for bad in ({"ws": 0}, {"ws": WS + 8}, {"nb": need - 1}):
        assert _attend(**bad) == b.SPECDEC_ERR_WORKSPACE, bad


def test_status_string():
    assert b.status_string(b.SPECDEC_ERR_NO_PAGES) == "not enough free pages"


def test_python_refuses_cpu_tensors():
    import target_model_verify_gb300 as tv
    tables = tv.alloc_page_tables(1, 2, 3, device="cpu")
    one = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(TypeError):
        tv.plan_pages(*tables, one, one, 16)
    pool = tv.alloc_paged_cache(2, 16, 4, 64, device="cpu")
    x = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        tv.append_paged(x, x, *pool, one.view(1, 1))
    with pytest.raises(TypeError):
        tv.verify_attention_paged(x, *pool, tables[0], one)


def test_plan_oracle_keeps_the_pages():
    """Every page is in one place, and a sequence's rows keep theirs from plan to plan."""
    r = random.Random(1)
    B, page, n_pages = 5, 16, 40
    state = ([[-1] * 20 for _ in range(B)], [0] * B, list(range(n_pages)), n_pages)
    lens = [0] * B
    for _ in range(200):
        start = [min(x, r.randint(0, 300)) if r.random() < 0.5 else x for x in lens]
        counts = [r.randint(0, min(20, 320 - s)) for s in start]
        before = [row[:h] for row, h in zip(state[0], state[1])]
        *state, slots, status = op.plan(*state, start, counts, page, n=20)
        if status == op.NO_PAGES:
            assert set(slots) == {-1} and sum(-(-(s + c) // page) for s, c in zip(start, counts)) > n_pages
            continue
        lens = [s + c for s, c in zip(start, counts)]
        used = [p for row, h in zip(state[0], state[1]) for p in row[:h]] + state[2][:state[3]]
        assert sorted(used) == list(range(n_pages))
        for b_, row in enumerate(state[0]):
            h = state[1][b_]
            assert h == -(-lens[b_] // page) and row[:min(h, len(before[b_]))] == before[b_][:h]
            for i in range(counts[b_]):
                at = start[b_] + i
                assert slots[b_ * 20 + i] == row[at // page] * page + at % page
    real = [s for s in slots if s >= 0]
    assert len(set(real)) == len(real)


def test_gather_oracle():
    pages = np.arange(3 * 16 * 2 * 1, dtype=float).reshape(3, 16, 2, 1)
    got = op.gather(pages, [2, -1, 0], 35)
    assert (got[:16] == pages[2]).all() and not got[16:32].any() and (got[32:] == pages[0, :3]).all()
