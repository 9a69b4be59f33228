"""What the bounds of the cache attention (tests/cache_bounds.py) rest on, without a GPU."""
import numpy as np
import pytest
import torch

from tests import cache_bounds as cb


def _e5m2(x):
    return x.to(torch.float8_e5m2)


def test_four_e5m2_terms_hold_every_f16_weight():
    """p = t0 + t1 / 8 + t2 / 64 + t3 / 512 for every f16 value up to 2^15, the terms e5m2 roundings
    of what the ones before leave, times 8; no term passes 2^15."""
    h = torch.arange(0x7801, dtype=torch.int32).to(torch.int16).view(torch.float16)
    assert h[-1] == 2.0 ** 15
    rest, total = h.clone(), torch.zeros(len(h), dtype=torch.float64)
    for t in range(4):
        term = _e5m2(rest)
        assert term.double().abs().max() <= 2.0 ** 15
        total += term.double() / 8.0 ** t
        rest = (rest - term.to(torch.float16)) * 8
    assert torch.equal(total, h.double())
    # an e5m2 code is the upper byte of that f16 value
    term = _e5m2(h)
    np.testing.assert_array_equal(term.view(torch.uint8).numpy().astype(np.int64) << 8,
                                  term.to(torch.float16).view(torch.int16).numpy())


# The shapes of one sequence whose tiles are shared by many CTAs; 64 rows are the smallest block.
SHARED = [(2, 4, 1, 128, 20000), (2, 4, 2, 256, 9001), (40, 1, 1, 64, 5000), (9, 16, 2, 128, 4001), (3, 8, 8, 128, 33001)]


@pytest.mark.parametrize("kind", ["kv8", "masked"])
@pytest.mark.parametrize("n,Hq,Hkv,D,L", SHARED)
def test_no_run_of_rows_can_be_lost_unnoticed(kind, n, Hq, Hkv, D, L):
    """Leaving out any 64 rows (a partial that the merge drops holds more) moves some output by more
    than three times its bound."""
    q, k, v = cb.with_marks(np.random.default_rng([n, L]), n, Hq, Hkv, D, L)
    _, _, shows = cb.outputs_and_bounds(kind, q[:, :1], k[:, :1], v[:, :1], without=64)
    shows = shows[:(L - n) // 64]                # the rest is not seen by every position
    assert shows.min() > 3, (shows.min(), shows.argmin())


def test_two_e4m3_terms_of_a_query_row():
    """Every bf16 value under every largest element in [2^7, 2^8): exact from 2^-9 of that on, else off
    by at most 2^-17 of it, which occurs."""
    x = torch.arange(0x4380, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).double()    # 0 .. 2^8
    x = x[x < 256]
    e4m3 = lambda t: t.float().to(torch.float8_e4m3fn).double()                              # noqa: E731
    hi = e4m3(x)
    off = (x - hi - e4m3(x - hi)).abs()
    for largest in x[x >= 128].tolist():
        here = x <= largest
        assert not off[here & (x >= largest * 2.0 ** -9)].any()
        assert (off[here] <= 2.0 ** -17 * largest).all()
    assert off.max() == 2.0 ** -17 * 128 and float(x[off.argmax()]) < 1
