"""Plans of a paged cache at the ends of what they take, and of tables that hold what they should not."""
import pytest
import torch

from tests.test_gpu_paged_cache import _i

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("B", [2, 1100])                      # the rows with the gaps between them, and behind them
def test_the_largest_map(B):
    """Entries up to 2^31 - 6: sequences with few rows and none at its very end."""
    import target_model_verify_gb300 as tv
    rows = 2 ** 31 - 5
    tables = tv.alloc_page_tables(B, 2, 2 * B, device=DEV)
    cu = torch.full((B + 1,), rows - 3, dtype=torch.int32, device=DEV)
    cu[0], cu[1], cu[B] = 0, 2, rows
    if B == 2:
        cu[1] = rows - 3
    counts = torch.zeros(B, dtype=torch.int32, device=DEV)
    counts[0], counts[B - 1] = 2, 3
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    slots = tv.plan_pages(*tables, torch.full((B,), 15, dtype=torch.int32, device=DEV), counts, 16, n=rows, cu_rows=cu,
                          workspace=ws)
    assert tv.read_status(ws) == 0
    table = tables[0]
    first, last = table[0].tolist(), table[B - 1].tolist()
    assert slots[:2].tolist() == [first[0] * 16 + 15, first[1] * 16]
    assert slots[-3:].tolist() == [last[0] * 16 + 15, last[1] * 16, last[1] * 16 + 1]
    for part in slots[2:-3].split(1 << 28):
        assert (part == -1).all()
    assert tables[1].tolist() == [2] + [1] * (B - 2) + [2]
