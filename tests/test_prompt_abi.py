"""The prompt attention's calls check their arguments on the host before anything reaches a GPU (CPU)."""
import pytest
import torch

from target_model_verify_gb300 import _binding as b
from target_model_verify_gb300 import build as libbuild

P, WS, BIG = 4096, 4096 * 256, 1 << 30


@pytest.fixture(scope="module", autouse=True)
def _lib():
    libbuild.build()
    b.lib()


def _attend(q=P, qs=4096, k=P, ks=1024, v=P, vs=1024, cu=P, slopes=0, B=2, T=100, Hq=32, Hkv=8, D=128, scale=0.0,
            cap=0.0, window=0, out=P, ws=WS, nb=BIG):
    # Fake but aligned addresses: every check below fails before any access.
    return b.specdec_prompt_attention(q, qs, k, ks, v, vs, cu, slopes, B, T, Hq, Hkv, D, scale, cap, window, out, ws,
                                      nb, None)


def test_argument_errors():
    size = b.specdec_prompt_attention_workspace_size
    need = size(2, 100, 32, 8, 128)
    assert 512 <= need <= 1024
    assert size(2, 1 << 20, 32, 8, 128) >= 16 * (1 << 20) // 64
    assert _attend(B=0, q=0, ws=0) == b.SPECDEC_OK
    assert _attend(T=0, q=0, ws=0) == b.SPECDEC_OK
    for bad in ({"D": 96}, {"D": 0}, {"Hq": 30}, {"Hq": 4}, {"Hkv": 0}, {"B": -1}, {"T": -1}, {"T": (1 << 30) + 1},
                {"Hq": 129 * 8}, {"T": 1 << 30, "Hq": 8}, {"B": 1 << 28}, {"Hq": 1 << 21, "Hkv": 1 << 20}):
        assert _attend(**bad) == b.SPECDEC_ERR_UNSUPPORTED, bad
        shape = dict(B=2, T=100, Hq=32, Hkv=8, D=128)
        shape.update(bad)
        assert size(*(shape[x] for x in ("B", "T", "Hq", "Hkv", "D"))) == 0, bad
    for bad in ({"q": 0}, {"k": 0}, {"v": 0}, {"cu": 0}, {"out": 0}, {"q": P + 8}, {"k": P + 2}, {"v": P + 8},
                {"out": P + 2}, {"cu": P + 2}, {"slopes": P + 1}, {"qs": 4088}, {"qs": 4100}, {"ks": 1016},
                {"vs": 1028}, {"ks": 1 << 31}, {"vs": -1024}, {"scale": float("nan")}, {"scale": 1e-35},
                {"scale": 1e31}, {"cap": -1.0}, {"cap": 1e-35}, {"cap": 1001.0}, {"cap": float("inf")},
                {"window": -1}):
        assert _attend(**bad) == b.SPECDEC_ERR_INVALID_ARG, bad
    for bad in ({"ws": 0}, {"ws": WS + 8}, {"nb": need - 1}):
        assert _attend(**bad) == b.SPECDEC_ERR_WORKSPACE, bad


def test_python_refuses_cpu_tensors():
    import target_model_verify_gb300 as tv
    x = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        tv.prompt_attention(x, x, x, torch.tensor([0, 3], dtype=torch.int32))
