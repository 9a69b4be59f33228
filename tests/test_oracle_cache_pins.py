"""Pins of the fp64 oracle of the 8-bit cache and the masked attention (CPU)."""
import math

import numpy as np
import pytest
import torch

from oracle import attention as oa
from oracle import cache as oc


def test_e4m3_matches_torch():
    rng = np.random.default_rng(0)
    x = rng.normal(size=40000) * np.exp2(rng.integers(-12, 10, 40000))
    ties = oc.e4m3_values()
    x = np.concatenate([x, (ties[1:] + ties[:-1]) / 2, ties, [0.0, -0.0, 2.0 ** -10, 448.0]])
    t = torch.tensor(x, dtype=torch.float32).clamp(-448, 448)
    want = t.to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(oc.to_e4m3(t.double().numpy()), want)
    assert oc.to_e4m3(1e9) == 448 and oc.to_e4m3(-np.inf) == -448 and np.isnan(oc.to_e4m3(np.nan))


def test_block_scale():
    assert oc.block_scale(448.0) == 1 and oc.block_scale(448.1) == 2 and oc.block_scale(224.0) == 0.5
    assert oc.block_scale(0.0) == 2.0 ** -40 and oc.block_scale(1e38) == 2.0 ** 40


def test_append_keeps_the_values():
    """What is appended in pieces stands for the values within half a step, whatever the pieces."""
    rng = np.random.default_rng(1)
    x = rng.normal(size=(1, 70, 2, 64)) * np.exp(rng.normal(size=(1, 70, 1, 1)))
    whole = oc.append(x, np.zeros((1, 80, 2, 64)), np.zeros((1, 2, 3)), [5])
    codes, scales = np.zeros((1, 80, 2, 64)), np.zeros((1, 2, 3))
    for a, e in ((0, 3), (3, 27), (27, 60), (60, 70)):
        codes, scales = oc.append(x[:, a:e], codes, scales, [5 + a])
    np.testing.assert_array_equal(scales, whole[1])
    for c, s in ((codes, scales), whole):
        got = oc.dequantise(c, s)[:, 5:75]
        step = np.repeat(s, 32, axis=2)[:, :, 5:75].transpose(0, 2, 1)[..., None]
        # re-encoding rounds a second time only below the smallest normal code
        assert (np.abs(got - x) <= 2.0 ** -4 * np.abs(x) + 2 * 2.0 ** -10 * step).all()


def test_masked_attention_reduces_to_the_causal_form():
    rng = np.random.default_rng(2)
    q, k, v = rng.normal(size=(2, 3, 4, 8)), rng.normal(size=(2, 20, 2, 8)), rng.normal(size=(2, 20, 2, 8))
    want = oa.verify_attention(q, k, v, [20, 3])
    chain = dict(window=20, parent=(-1, 0, 1))
    for how in ({}, chain, {"slopes": np.zeros(4)}):
        np.testing.assert_allclose(oc.masked_attention(q, k, v, [20, 3], **how), want, rtol=1e-12)
    np.testing.assert_allclose(oc.masked_attention(q, k, v, [20, 3], softcap=1e6), want, rtol=1e-6)


def test_masked_attention_matches_torch_with_explicit_masks():
    rng = np.random.default_rng(3)
    n, L, parent = 5, 17, (-1, 0, 0, 1, 3)
    q, k, v = rng.normal(size=(1, n, 2, 8)), rng.normal(size=(1, L, 1, 8)), rng.normal(size=(1, L, 1, 8))
    depth = [0, 1, 1, 2, 3]
    up = {0: {0}, 1: {0, 1}, 2: {0, 2}, 3: {0, 1, 3}, 4: {0, 1, 3, 4}}
    slopes = [0.3, 0.7]
    bias = np.full((2, n, L), -math.inf)
    for i in range(n):
        for j in range(L):
            pj = j if j < L - n else L - n + depth[j - (L - n)]
            seen = j < L - n or (j - (L - n)) in up[i]
            away = L - n + depth[i] - pj
            if seen and away < 6:
                for h in range(2):
                    bias[h, i, j] = -slopes[h] * away
    t = lambda x: torch.tensor(x).transpose(1, 2)  # noqa: E731
    want = torch.nn.functional.scaled_dot_product_attention(
        t(q), t(k).expand(1, 2, L, 8), t(v).expand(1, 2, L, 8), attn_mask=torch.tensor(bias)[None])
    got = oc.masked_attention(q, k, v, [L], window=6, slopes=slopes, parent=parent)
    np.testing.assert_allclose(got, want.transpose(1, 2).numpy(), rtol=1e-10)


def test_one_visible_row_gives_its_value():
    rng = np.random.default_rng(4)
    q, k, v = rng.normal(size=(1, 3, 2, 8)), rng.normal(size=(1, 9, 2, 8)), rng.normal(size=(1, 9, 2, 8))
    got = oc.masked_attention(q, k, v, [9], window=1, softcap=2.0)
    np.testing.assert_allclose(got[0], v[0, 6:9], rtol=1e-12)
    assert not oc.masked_attention(q, k, v, [0]).any()


@pytest.mark.parametrize("planted", ["order", "depth"])
def test_planted_mistakes_show(planted):
    """A tree read as a chain, and node order taken for depth, differ from the definition."""
    rng = np.random.default_rng(5)
    q, k, v = rng.normal(size=(1, 3, 1, 8)), rng.normal(size=(1, 9, 1, 8)), rng.normal(size=(1, 9, 1, 8))
    right = oc.masked_attention(q, k, v, [9], parent=(-1, 0, 0), slopes=[1.0])
    if planted == "order":
        wrong = oc.masked_attention(q, k, v, [9], parent=(-1, 0, 1), slopes=[1.0])
    else:
        wrong = oc.masked_attention(q, k, v, [9], parent=(-1, 0, 0), slopes=[1.1])
    assert np.abs(right - wrong)[0, 2].max() > 1e-3
