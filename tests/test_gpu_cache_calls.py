"""What the cache operators' calls promise at their edges, on the GPU: tables that end early, options at
the ends of their ranges, workspaces, many query heads per KV head."""
import numpy as np
import pytest
import torch

from oracle import cache as oc

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
