"""Rows that a position does not see never reach its output, whatever they hold and whatever is done to the
scores beside them (caps, biases, windows, trees): outputs with NaN or infinities in such rows equal, bit for
bit, those without."""
import pytest
import torch

from tests.test_gpu_cache_attention import TREE26
from tests.test_gpu_paged_attention import _call as _call_paged
from tests.test_gpu_paged_attention import _inputs as _paged_inputs
from tests.test_gpu_prompt_attention import _call, _inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN, INF = float("nan"), float("inf")

HOW = pytest.mark.parametrize("how", [
    {}, {"softcap": 5.0}, {"softcap": 30.0, "window": 36}, {"softcap": 30.0, "window": 37}, {"window": 37},
    {"softcap": 20.0, "slopes": True}, {"softcap": 20.0, "slopes": True, "window": 37}, {"slopes": True},
], ids=str)


def _with_slopes(how, heads):
    how = dict(how)
    if how.get("slopes"):
        how["slopes"] = torch.exp2(-torch.arange(1, heads + 1, device=DEV, dtype=torch.float32))
    return how


@pytest.mark.parametrize("D", [64, 128, 256])
@HOW
@pytest.mark.parametrize("key,value", [(NAN, INF), (INF, NAN), (-INF, -INF)], ids=str)
def test_prompts_see_no_other_row(D, how, key, value):
    """In the sequences around one, in rows of no sequence and in later rows of its own; the last row seen
    has an odd distance from the block's first, and an even one."""
    how = _with_slopes(how, 4)
    q, k, v, cu = _inputs(40, [131, 201, 71], 4, 2, D, gaps=True)
    lo, hi = cu[1], cu[2]
    want = _call(q, k, v, cu, **how)
    for tail in (161, 160, 201):                              # of its own rows the first that is not clean
        qd, kd, vd = q.clone(), k.clone(), v.clone()
        qd[:lo] = qd[hi:] = NAN
        kd[:lo] = kd[lo + tail:] = key
        vd[:lo] = vd[lo + tail:] = value
        got = _call(qd, kd, vd, cu, **how)
        assert torch.equal(got[lo:lo + tail], want[lo:lo + tail])
        assert not got[lo + tail:hi].isfinite().any()         # they see their own


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("L", [1, 2, 7, 63, 64, 65, 127, 129, 255, 257])
def test_prompts_see_no_padding(D, L):
    """What a longer buffer holds behind the last sequence."""
    q, k, v, cu = _inputs(41, [L], 4, 2, D, gaps=True)
    for how in ({}, {"softcap": 30.0}, {"softcap": 30.0, "window": 20}):
        want = _call(q, k, v, cu, **how)
        for t in (k, v):
            t[:cu[0]] = t[cu[1]:] = NAN
        assert torch.equal(_call(q, k, v, cu, **how)[cu[0]:cu[1]], want[cu[0]:cu[1]])
        for t in (k, v):
            t[:cu[0]] = t[cu[1]:] = 1.0


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("how", [{}, {"softcap": 30.0}, {"softcap": 30.0, "slopes": True}], ids=str)
@pytest.mark.parametrize("window", [36, 37, 130])
@pytest.mark.parametrize("row", [20, 21])
def test_prompts_see_nothing_behind_the_window(D, how, window, row):
    """One row of a prompt is not clean: the positions whose window it has left are as without it."""
    how = dict(_with_slopes(how, 4), window=window)
    q, k, v, cu = _inputs(42, [300], 4, 2, D)
    want = _call(q, k, v, cu, **how)
    k[row] = v[row] = NAN
    got = _call(q, k, v, cu, **how)
    for part in (slice(0, row), slice(row + window, 300)):
        assert torch.equal(got[part], want[part])
    assert got[row:row + window].isnan().all()


# 2 query heads per KV head: 8 new positions go to the form for little work, 26 to the other
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [8, 26])
@pytest.mark.parametrize("how", [{}, {"softcap": 20.0}, {"softcap": 20.0, "slopes": True}, {"softcap": 20.0, "window": 33}],
                         ids=str)
def test_trees_over_pages_see_no_other_branch(D, n, how):
    """A node's row that is not clean reaches its descendants alone; one that the window has left, nobody."""
    how = _with_slopes(how, 4)
    L, node = 150, 3
    q, pages, table, lens = _paged_inputs(43, 1, n, 4, 2, D, 16, 10, [L])
    parent = TREE26[:n]
    want = _call_paged(q, pages, table, lens, parent=parent, **how)
    below = [False] * n
    for i in range(n):
        below[i] = i == node or (i > node and below[parent[i]])
    rows = [L - n + node] + ([L - n - how["window"]] if "window" in how else [])
    for t in pages:
        for row in rows:
            t[table[0, row // 16], row % 16] = NAN
    got = _call_paged(q, pages, table, lens, parent=parent, **how)
    for i in range(n):
        assert got[0, i].isnan().all() if below[i] else torch.equal(got[0, i], want[0, i]), i
