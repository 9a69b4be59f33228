"""Limits of the cache attention's options, refused on the host (CPU)."""
import pytest

from target_model_verify_gb300 import _binding as b
from tests.test_cache_abi import _attend, _lib  # noqa: F401  (the fixture builds and loads the library)


@pytest.mark.parametrize("name", ["specdec_verify_attention_kv8", "specdec_verify_attention_masked"])
def test_scales_that_leave_fp32(name):
    fn = getattr(b, name)
    for bad in ({"scale": 1.1e30}, {"scale": 3e38}, {"scale": 1.4e-45}, {"cap": 1.4e-45}):
        assert _attend(fn, **bad) == b.SPECDEC_ERR_INVALID_ARG, bad
    # what is allowed gets as far as the workspace
    for good in ({"scale": 1e30}, {"scale": 1.01e-30}, {"scale": -1.0}, {"cap": 1000.0}, {"cap": 1.01e-30}):
        assert _attend(fn, ws=0, **good) == b.SPECDEC_ERR_WORKSPACE, good
