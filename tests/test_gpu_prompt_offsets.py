"""Offsets of packed prompts that change while prompt_attention runs: outputs may be any, but only rows of the
batch are read and written, and items that do not lie in it are passed over without a trace.

The offsets change at a known place here: they stand in the workspace, where the kernel that lists the items
writes how many there are and which is next. It counts items of what the test put there, and finds no sequence
when it comes to write the list, whose place the test has filled beforehand."""
import pytest
import torch

from tests.test_gpu_prompt_attention import _i

pytestmark = pytest.mark.gpu
DEV = "cuda"
COUNT, LIST = 256, 512                        # of the workspace: number of items and next one; the list


def _listed(D, G, entries, T, q, k, v, out):
    """The call with `entries` as its list; (status, what lies behind the workspace is as it was)."""
    import target_model_verify_gb300 as tv
    from target_model_verify_gb300 import _binding as b
    size = tv.prompt_attention_workspace_bytes(1, T, G, 1, D)
    big = torch.full((size + 4096,), 0x5a, dtype=torch.uint8, device=DEV)
    ws = big[:size]
    assert ws.data_ptr() % 256 == 0
    ws[COUNT:COUNT + 8].view(torch.int32).copy_(_i([0, T]))
    at = ws[LIST:LIST + 16 * len(entries)]
    at.view(torch.int32).copy_(_i(entries).flatten())
    rc = b.specdec_prompt_attention(q.data_ptr(), G * D, k.data_ptr(), D, v.data_ptr(), D, ws.data_ptr() + COUNT, 0, 1,
                                    T, G, 1, D, 0.0, 0.0, 0, out.data_ptr(), ws.data_ptr(), size,
                                    torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    status = tv.read_status(ws)
    assert (big[size:] == 0x5a).all()
    return status


@pytest.mark.parametrize("D", [64, 128, 256])
def test_items_outside_the_batch_are_passed_over(D):
    """Every CTA begins with an item that is none, and goes on to sequences' own."""
    import target_model_verify_gb300 as tv
    G = 2
    span = 64 * (2 if D <= 128 else 1)                    # tokens of an item
    N = 400                                               # items of one sequence of all rows
    T = N * span
    g = torch.Generator(device=DEV).manual_seed(D)
    q, k, v = (torch.randn(T, h, D, generator=g, device=DEV).to(torch.bfloat16) for h in (G, 1, 1))
    # sequences of 150 rows, 50 between them: all items of the former
    top = 2 ** 31 - 1
    odd = [(0, 0, 0, 0), (-1, 0, 10, 0), (T, 0, 1, 0), (T - 5, 0, 10, 0), (5, 10, 10, 0), (5, -3, 10, 0),
           (top, 0, top, 0), (0, 0, -7, 0), (0, top, top, 0), (-top - 1, -top - 1, -top - 1, 0), (0x5a5a5a5a,) * 4]
    entries = [odd[i % len(odd)] for i in range(160)]
    cu, seqs, starts = [0], [], range(0, 150, span)
    while len(entries) + len(starts) <= N:
        entries += [(cu[-1], t0, 150, 0) for t0 in starts]
        seqs.append(cu[-1])
        cu += [cu[-1] + 150, cu[-1] + 200]
    entries += [odd[0]] * (N - len(entries))
    want = tv.prompt_attention(q, k, v, _i(cu))
    out = torch.full_like(q, 7.0)
    assert _listed(D, G, entries, T, q, k, v, out) == 0
    left = torch.ones(T, dtype=torch.bool, device=DEV)
    for row in seqs:
        assert torch.equal(out[row:row + 150], want[row:row + 150]), row
        left[row:row + 150] = False
    assert (out[left] == 7).all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_list_of_nothing(D):
    """What an earlier call left in the workspace in place of every item."""
    G, T = 1, 400 * 128 * (2 if D <= 128 else 1)
    q, k, v = (torch.zeros(T, 1, D, dtype=torch.bfloat16, device=DEV) for _ in range(3))
    out = torch.full_like(q, 7.0)
    assert _listed(D, G, [(0x5a5a5a5a,) * 4] * 400, T, q, k, v, out) == 0
    assert (out == 7).all()
