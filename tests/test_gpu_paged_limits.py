"""Plans of a paged cache at the ends of what they take, and of tables that hold what they should not."""
import random

import pytest
import torch

from oracle import paged as op
from tests.test_gpu_paged_cache import Batch, _i

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


@pytest.mark.parametrize("max_pages", [8, 9000])              # one CTA, and a cluster
@pytest.mark.parametrize("entry", [-1, 40, 2 ** 31 - 1])
def test_entries_that_are_no_pages_are_told(entry, max_pages):
    """They go onto the stack and off it again as pages would; the status word says so each time, with a map
    and without, and not of a plan that moves others."""
    batch = Batch(3, max_pages, 40, 16)
    batch.plan([0, 0, 0], [40, 30, 50])
    batch.gpu[0][1, 1] = entry
    batch.load()
    batch.plan([40, 0, 50], [20, 20, 0], n=20, expect=op.INVALID)      # a row on it
    batch.plan([60, 0, 50], [0, 32, 0], n=32, expect=op.INVALID)
    batch.plan([0, 0, 50], [35, 20, 0])                                # it stays where it is
    batch.plan([0, 0, 50], [35, 16, 0], expect=op.INVALID)             # given back
    batch.plan([35, 16, 50], [0, 0, 16], expect=op.INVALID)            # taken again
    batch.plan([35, 16, 0], [0, 0, 66])                                # it stays there
    batch.plan([0, 0, 0], [0, 0, 0], expect=op.INVALID)


def test_two_pools_hold_all_their_pages_after_many_plans():
    """Steps and admissions of two batches in turn: no page is lost, and none is in two places."""
    r = random.Random(3)
    batches = [Batch(B, 40, pages, 16) for B, pages in ((5, 100), (300, 2000))]
    for step in range(60):
        for batch in batches:
            B, pages = batch.gpu[0].shape[0], batch.gpu[2].shape[0]
            lens = [r.randint(0, 400) if r.random() < 0.6 else 0 for _ in range(B)]
            while sum(-(-x // 16) for x in lens) > pages:
                lens[r.randrange(B)] = 0
            batch.plan([0] * B, lens, **({} if step % 3 else {"n": 400}))
            table, held, free, n_free = batch.host
            there = [p for row, h in zip(table, held) for p in row[:h]] + free[:n_free]
            assert sorted(there) == list(range(pages))


@pytest.mark.parametrize("at", [1, 2, 3])
@pytest.mark.parametrize("B,n", [(3, 5), (40, 130)])          # one CTA, and a cluster
def test_maps_at_any_entry(at, B, n):
    """A map that does not begin on 16 bytes is filled, and read, as any; what is around it stays."""
    import target_model_verify_gb300 as tv
    batch = Batch(B, 12, 10 * B, 16)
    big = torch.full((B * n + 8,), 77, dtype=torch.int32, device=DEV)
    slots = big[at:at + B * n].view(B, n)
    counts = [n - b % 3 for b in range(B)]
    *_, want, status = op.plan(*batch.host, [7] * B, counts, 16, n)
    tv.plan_pages(*batch.gpu, _i([7] * B), _i(counts), 16, slots=slots, workspace=batch.ws)
    assert tv.read_status(batch.ws) == status == op.OK
    assert slots.flatten().tolist() == want
    assert (big[:at] == 77).all() and (big[at + B * n:] == 77).all()
    new = [torch.randn(B, n, 2, 64, device=DEV).to(torch.bfloat16) for _ in range(2)]
    pool = tv.alloc_paged_cache(10 * B, 16, 2, 64, device=DEV)
    tv.append_paged(*new, *pool, slots, workspace=batch.ws)
    assert tv.read_status(batch.ws) == op.OK
    live = slots.flatten() >= 0
    for t, x in zip(pool, new):
        assert torch.equal(t.view(-1, 2, 64)[slots.flatten()[live].long()], x.view(-1, 2, 64)[live])
