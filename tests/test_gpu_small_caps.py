"""Caps and scales at the ends of what the attentions take: scores of exactly 0 stay 0.

A cap of at most 1e-8 leaves scores that differ by 2e-8 at most, and so weights that differ by as much:
the output is the mean of the values seen, rounded to bf16, to the weights' rounding (2^-8 of each)."""
import pytest
import torch

from tests.test_gpu_prompt_attention import _i

pytestmark = pytest.mark.gpu
DEV = "cuda"
ENDS = pytest.mark.parametrize("scale,cap", [(1e30, 1e-30), (1e30, 1e-9), (1e10, 1e-30), (1.0, 1e-30), (1e-30, 1e-30),
                                             (1e-30, 1e-8)])


def _qkv(D):
    g = torch.Generator(device=DEV).manual_seed(D)
    q, k, v = (torch.randn(100, h, D, generator=g, device=DEV).to(torch.bfloat16) for h in (4, 2, 2))
    q[::2] = 0                                            # every score of these is 0
    k[40:60] = 0                                          # and with these
    mean = v.double().cumsum(0) / torch.arange(1, 101, device=DEV)[:, None, None]
    spread = v.double().abs().cumsum(0) / torch.arange(1, 101, device=DEV)[:, None, None]
    return q, k, v, *(t.repeat_interleave(2, dim=1) for t in (mean, spread))


def _close(out, mean, spread):
    assert ((out.double() - mean).abs() <= (2.0 ** -8 * (mean.abs() + spread) + 1e-6) * (1 + 2.0 ** -7)).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@ENDS
def test_prompts(D, scale, cap):
    import target_model_verify_gb300 as tv
    q, k, v, mean, spread = _qkv(D)
    _close(tv.prompt_attention(q, k, v, _i([0, 100]), scale=scale, softcap=cap), mean, spread)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [8, 9])                     # 16 rows and 18: both forms over pages
@ENDS
def test_caches(D, n, scale, cap):
    import target_model_verify_gb300 as tv
    q, k, v, mean, spread = _qkv(D)
    pages = [torch.zeros(7, 16, 2, D, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    for t, x in zip(pages, (k, v)):
        t.view(-1, 2, D)[:100] = x
    new, lens = q[None, -n:].contiguous(), _i([100])
    for out in (tv.verify_attention_paged(new, *pages, _i([list(range(7))]), lens, scale=scale, softcap=cap),
                tv.verify_attention_masked(new, k[None].contiguous(), v[None].contiguous(), lens, scale=scale, softcap=cap)):
        _close(out[0], mean[-n:], spread[-n:])
