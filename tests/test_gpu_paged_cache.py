"""Page tables, slot maps and rows of a paged cache on the GPU (plan_pages, append_paged)
against plain Python (oracle/paged.py). Whole numbers and copies: equality throughout."""
import random

import pytest
import torch

from oracle import paged as op

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _i(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Batch:
    """The tables on both sides."""

    def __init__(self, B, max_pages, n_pages, page):
        import target_model_verify_gb300 as tv
        self.tv, self.page = tv, page
        self.gpu = tv.alloc_page_tables(B, max_pages, n_pages, device=DEV)
        self.ws = torch.empty(256, dtype=torch.uint8, device=DEV)
        self.load()

    def load(self):
        table, held, free, n_free = self.gpu
        self.host = (table.tolist(), held.tolist(), free.tolist(), n_free.item())

    def plan(self, start, counts, n=None, cu_rows=None, n_slots=None, expect=op.OK):
        *self.host, want, status = op.plan(*self.host, start, counts, self.page, n, cu_rows, n_slots)
        got = self.tv.plan_pages(*self.gpu, _i(start), _i(counts), self.page, n=n if cu_rows is None else n_slots,
                                 cu_rows=None if cu_rows is None else _i(cu_rows), workspace=self.ws)
        assert self.tv.read_status(self.ws) == status == expect
        table, held, free, n_free = self.gpu
        assert table.tolist() == self.host[0]
        assert held.tolist() == self.host[1]
        assert free.tolist() == self.host[2]
        assert n_free.item() == self.host[3]
        assert (got is None) == (want is None)
        if want is not None:
            assert got.flatten().tolist() == want
            assert got.shape == ((len(start), n) if cu_rows is None else (n_slots,))
        return got


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_steps_of_a_batch(page):
    """Admission, steps with rejected drafts, requests that end and others in their place."""
    r = random.Random(page)
    B, n = 7, 5
    batch = Batch(B, 5 * 256 // page, 4 * B * 256 // page, page)
    lens = [0] * B
    for step in range(25):
        for b in range(B):
            if lens[b] == 0 or lens[b] > 3 * 256:
                lens[b] = r.randint(1, 2 * 256) if r.random() < 0.7 else 0
                if step == 0 and b == 1:
                    lens[b] = page                     # whole pages
                batch.plan([lens[x] if x != b else 0 for x in range(B)], [0 if x != b else lens[b] for x in range(B)],
                           cu_rows=[0 if x <= b else lens[b] for x in range(B + 1)], n_slots=lens[b])
        live = [n if lens[b] else 0 for b in range(B)]
        batch.plan(lens, live, n=n)
        kept = [r.randint(1, n) if lens[b] else 0 for b in range(B)]
        batch.plan(lens, kept, n=n if step % 2 else None)
        lens = [lens[b] + kept[b] for b in range(B)]
    batch.plan([0] * B, [0] * B)
    assert batch.gpu[3].item() == 4 * B * 256 // page and batch.gpu[1].sum().item() == 0
    assert sorted(batch.gpu[2].tolist()) == list(range(4 * B * 256 // page))


@pytest.mark.parametrize("B,most,page", [(1, 1, 16), (3, 5000, 16), (40, 700, 32), (1030, 9, 16), (2100, 40, 16),
                                         (33, 1, 256)])
def test_packed_prompts(B, most, page):
    """Many sequences and many rows: one CTA and a cluster, several chunks of sequences; gaps in the map."""
    r = random.Random(B)
    lens = [r.randint(0, most) if b % 5 else most for b in range(B)]
    gap = [r.randint(0, 2) for _ in range(B + 1)]
    cu = [gap[0]]
    for b in range(B):
        cu.append(cu[-1] + lens[b] + gap[b + 1])
    pages = -(-most // page)
    batch = Batch(B, pages + 2, B * pages + 1, page)
    batch.plan([0] * B, lens, cu_rows=cu, n_slots=cu[-1] + 3)
    batch.plan([0] * B, [x // 2 for x in lens])                                  # half of them given back
    batch.plan([x // 3 for x in lens], [x - x // 3 for x in lens], cu_rows=cu, n_slots=cu[-1])
    batch.plan([0] * B, [0] * B, cu_rows=cu, n_slots=cu[-1])
    assert batch.gpu[3].item() == B * pages + 1


def test_what_is_given_back_serves_the_same_call():
    """Requests that end and requests that begin in one plan, with no page to spare."""
    batch = Batch(4, 8, 12, 16)
    batch.plan([0] * 4, [100, 80, 0, 0], n=100)
    assert batch.gpu[3].item() == 0
    batch.plan([0] * 4, [0, 0, 90, 96], n=100)
    assert batch.gpu[3].item() == 0


@pytest.mark.parametrize("B,page", [(300, 16), (1500, 16), (40, 32)])
def test_a_cluster_gives_and_takes_at_once(B, page):
    """Requests that shrink, end, stay, grow and begin, in one plan with a map of many rows."""
    r = random.Random(B)
    most = 6 * page
    batch = Batch(B, 7, 4 * B, page)
    lens = [r.randint(0, most) if b % 2 else 0 for b in range(B)]
    while sum(-(-x // page) for x in lens) > 4 * B:
        lens[r.randrange(B)] = 0
    batch.plan([0] * B, lens)
    for _ in range(3):
        start = [r.choice((0, x, x // 2)) for x in lens]
        counts = [r.choice((0, 1, r.randint(0, most - s))) for s in start]
        cu = [0]
        for c in counts:
            cu.append(cu[-1] + c + r.randint(0, 1))
        while sum(-(-(s + c) // page) for s, c in zip(start, counts)) > 4 * B:
            b = r.randrange(B)
            start[b] = counts[b] = 0
        batch.plan(start, counts, cu_rows=cu, n_slots=cu[-1])
        lens = [s + c for s, c in zip(start, counts)]


def test_too_few_pages_change_nothing():
    batch = Batch(3, 8, 9, 16)
    batch.plan([0, 0, 0], [33, 40, 16], n=40)
    batch.plan([33, 40, 16], [10, 10, 40], n=40, expect=op.NO_PAGES)
    batch.plan([33, 40, 16], [10, 10, 20], n=40, expect=op.NO_PAGES)      # 3 + 4 + 3 pages of 9
    batch.plan([33, 40, 16], [10, 10, 16], n=40)                          # 3 + 4 + 2


def test_lengths_that_ask_for_more_than_32_bits_of_pages():
    import target_model_verify_gb300 as tv
    B = 33                                            # 33 * 2^26 pages
    tables = tv.alloc_page_tables(B, 1 << 26, 4, device=DEV)
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    tv.plan_pages(*tables, _i([0] * B), _i([1 << 30] * B), 16, workspace=ws)
    assert tv.read_status(ws) == op.NO_PAGES
    assert tables[3].item() == 4 and not tables[1].any() and (tables[0][:, :9] == -1).all()


def test_impossible_sequences_are_left():
    batch = Batch(6, 4, 30, 16)
    batch.plan([0] * 6, [40, 30, 20, 64, 1, 0], n=64)
    batch.plan([-1, 30, 20, 60, 2 ** 31 - 1, 0], [5, -2, 5, 5, 5, 6], n=5, expect=op.INVALID)
    batch.plan([40, 30, 25, 64, 1, 5], [0, 5, 2 ** 31 - 1, 0, 3, 0], n=5, expect=op.INVALID)
    for cu in ([0, 1, 2, 3, 4, 5, 6], [-1, 5, 10, 15, 20, 25, 30], [0, 5, 3, 15, 20, 25, 30],
               [0, 5, 10, 15, 20, 25, 31], [0, 5, 10, 2 ** 31 - 1, 20, 25, 30]):
        batch.plan([10, 10, 10, 10, 10, 10], [5, 5, 5, 0, 5, 5], cu_rows=cu, n_slots=30, expect=op.INVALID)


def test_bad_state_is_refused_on_the_device():
    """Counts of pages held and free that cannot be."""
    for held, n_free in (([5, 1], 3), ([-1, 1], 3), ([2, 1], 7), ([2, 1], -1), ([2, 1], 6)):
        batch = Batch(2, 4, 6, 16)
        batch.plan([0, 0], [30, 16])
        batch.gpu[1].copy_(_i(held))
        batch.gpu[3].fill_(n_free)
        batch.load()
        batch.plan([0, 0], [16, 16], n=16, expect=op.INVALID)
    batch = Batch(2, 4, 6, 16)
    batch.plan([0, 0], [30, 16])
    for entry in (-1, 6, 2 ** 31 - 1):
        batch.gpu[0][0, 1] = entry
        batch.load()
        batch.plan([15, 10], [5, 5], n=5, expect=op.INVALID)


def test_empty_batches_and_maps():
    import target_model_verify_gb300 as tv
    tables = tv.alloc_page_tables(0, 4, 6, device=DEV)
    none = _i([])
    assert tv.plan_pages(*tables, none, none, 16) is None
    assert tv.plan_pages(*tables, none, none, 16, n=3).shape == (0, 3)
    got = tv.plan_pages(*tables, none, none, 16, n=5, cu_rows=_i([0]))
    assert got.tolist() == [-1] * 5
    batch = Batch(2, 4, 6, 16)
    batch.plan([3, 0], [0, 0], n=0)
    batch.plan([3, 0], [1, 0], n=0, expect=op.INVALID)
    batch.plan([3, 0], [0, 0], cu_rows=[0, 0, 0], n_slots=0)


def test_captured_plan_and_append():
    """A step's plan and append in a graph, replayed on new lengths."""
    import target_model_verify_gb300 as tv
    B, n, page, H, D = 3, 4, 16, 2, 64
    batch = Batch(B, 8, 20, page)
    g = torch.Generator(device=DEV).manual_seed(1)
    new = [torch.randn(B, n, H, D, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2)]
    pool = tv.alloc_paged_cache(20, page, H, D, device=DEV)
    for t in pool:
        t.zero_()
    start, counts = _i([0, 0, 0]), _i([n] * B)
    ws = [torch.empty(256, dtype=torch.uint8, device=DEV) for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        slots = tv.plan_pages(*batch.gpu, start, counts, page, n=n, workspace=ws[0])
        tv.append_paged(*new, *pool, slots, workspace=ws[1])
    want = [t.clone() for t in pool]
    for step in range(6):
        start.copy_(_i([step * n, 7 * step, 3 * step]))
        new[0].mul_(-1)
        *batch.host, m, status = op.plan(*batch.host, start.tolist(), [n] * B, page, n)
        graph.replay()
        assert status == 0 and tv.read_status(ws[0]) == 0 and tv.read_status(ws[1]) == 0
        assert slots.flatten().tolist() == m and batch.gpu[0].tolist() == batch.host[0]
        for x in (0, 1):
            want[x].view(-1, H, D)[slots.flatten().long()] = new[x].view(-1, H, D)
            assert torch.equal(pool[x], want[x])


# ------------------------------------------------------------------ rows --

def _pool(g, n_pages, page, H, D):
    return [torch.randn(n_pages, page, H, D, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2)]


def _append_and_check(new, pool, slots, rows=None, expect=0):
    import target_model_verify_gb300 as tv
    want = [t.clone() for t in pool]
    H, D = pool[0].shape[2:]
    total, per = pool[0].shape[0] * pool[0].shape[1], new[0].shape[1] if new[0].dim() == 4 else new[0].shape[0]
    for i, s in enumerate(slots.flatten().tolist()):
        src = i if rows is None else rows.flatten()[i].item() + i // per * per
        if 0 <= s < total and (rows is None or 0 <= rows.flatten()[i].item() < per):
            for x in (0, 1):
                want[x].view(-1, H, D)[s] = new[x].reshape(-1, H, D)[src]
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    got = tv.append_paged(*new, *pool, slots, rows=rows, workspace=ws)
    assert tv.read_status(ws) == expect
    for x in (0, 1):
        assert got[x] is pool[x] and torch.equal(pool[x], want[x])


@pytest.mark.parametrize("H,D", [(1, 64), (3, 64), (1, 128), (8, 128), (5, 256), (17, 128)])
@pytest.mark.parametrize("B,n,page", [(1, 1, 16), (3, 5, 32), (2, 130, 256)])
def test_append_copies_rows(H, D, B, n, page):
    g = torch.Generator(device=DEV).manual_seed(H * D + n)
    pool = _pool(g, 3 + B * n // page, page, H, D)
    kv = torch.randn(B, n, 2, H, D, generator=g, device=DEV).to(torch.bfloat16)
    slots = torch.randperm(pool[0].shape[0] * page, generator=g, device=DEV)[:B * n].to(torch.int32).view(B, n)
    slots[0, n // 2] = -1
    _append_and_check(list(kv.unbind(2)), pool, slots)
    packed = [t.reshape(-1, 2, H, D)[:, 0] for t in (kv, kv.flip(0))]           # a packed batch's slices
    _append_and_check(packed, pool, slots.flatten())
    rows = torch.randint(0, n, (B, n), generator=g, device=DEV).to(torch.int32)
    rows[0, n // 2] = -7                                                        # not read
    _append_and_check(list(kv.unbind(2)), pool, slots, rows)


def test_append_skips_what_does_not_fit():
    g = torch.Generator(device=DEV).manual_seed(2)
    pool = _pool(g, 4, 16, 2, 64)
    new = [torch.randn(2, 3, 2, 64, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2)]
    _append_and_check(new, pool, _i([[0, 64, 1], [-2, 2, 2 ** 31 - 1]]), expect=op.INVALID)
    _append_and_check(new, pool, _i([[0, 5, 1], [7, 2, 63]]), _i([[0, 3, 1], [-1, 2, 0]]), expect=op.INVALID)
    _append_and_check(new, pool, _i([[0, 5, 1], [7, 2, 63]]))


def test_append_of_nothing():
    import target_model_verify_gb300 as tv
    pool = tv.alloc_paged_cache(2, 16, 2, 64, device=DEV)
    for shape in ((0, 3), (2, 0), (0,)):
        new = torch.empty(*shape, 2, 64, dtype=torch.bfloat16, device=DEV)
        tv.append_paged(new, new, *pool, torch.empty(shape, dtype=torch.int32, device=DEV))
