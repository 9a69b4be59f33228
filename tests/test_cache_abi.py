"""The 8-bit cache's and the masked attention's calls check their arguments on
the host before anything reaches a GPU (CPU)."""
import ctypes

import pytest
import torch

from target_model_verify_gb300 import _binding as b
from target_model_verify_gb300 import build as libbuild

P, WS, BIG = 4096, 4096 * 256, 1 << 30


@pytest.fixture(scope="module", autouse=True)
def _lib():
    libbuild.build()
    b.lib()


def _append(k=P, ks=1024, v=P, vs=1024, start=P, counts=0, rows=0, B=1, n=5, H=8, D=128, Lmax=64,
            kc=P, vc=P, sk=P, sv=P, ws=WS, nb=BIG):
    # Fake but aligned addresses: every check below fails before any access.
    return b.specdec_kv8_append(k, ks, v, vs, start, counts, rows, B, n, H, D, Lmax, kc, vc, sk, sv, ws, nb,
                                None)


def test_append_argument_errors():
    assert b.specdec_kv8_append_workspace_size() == 256
    assert _append(B=0, k=0, ws=0) == b.SPECDEC_OK                     # empty batch: no-op
    for bad in ({"D": 96}, {"D": 0}, {"n": 0}, {"H": 0}, {"B": -1}, {"Lmax": 0}, {"Lmax": (1 << 30) + 1},
                {"B": 1 << 20, "Lmax": 1 << 20, "H": 1024}, {"B": 1 << 20, "n": 1 << 20}):
        assert _append(**bad) == b.SPECDEC_ERR_UNSUPPORTED, bad
    for bad in ({"k": 0}, {"v": 0}, {"start": 0}, {"kc": 0}, {"vc": 0}, {"sk": 0}, {"sv": 0}, {"k": P + 2},
                {"vc": P + 8}, {"sk": P + 2}, {"counts": P + 1}, {"rows": P + 2}, {"ks": 1016}, {"vs": 1028},
                {"ks": -1024}):
        assert _append(**bad) == b.SPECDEC_ERR_INVALID_ARG, bad
    for bad in ({"ws": 0}, {"ws": WS + 8}, {"nb": 255}):
        assert _append(**bad) == b.SPECDEC_ERR_WORKSPACE, bad


def _attend(fn, q=P, qs=4096, kc=P, vc=P, sk=P, sv=P, lens=P, parent=None, slopes=0, B=1, n=5, Hq=32, H=8,
            D=128, Lmax=64, scale=0.0, cap=0.0, window=0, out=P, ws=WS, nb=BIG):
    par = 0 if parent is None else ctypes.addressof((ctypes.c_int32 * len(parent))(*parent))
    scales = (sk, sv) if fn is b.specdec_verify_attention_kv8 else ()
    return fn(q, qs, kc, vc, *scales, lens, par, slopes, B, n, Hq, H, D, Lmax, scale, cap, window, out, ws, nb,
              None)


@pytest.mark.parametrize("name", ["specdec_verify_attention_kv8", "specdec_verify_attention_masked"])
def test_attention_argument_errors(name):
    fn, size = getattr(b, name), getattr(b, name + "_workspace_size")
    need = size(1, 5, 32, 8, 128, 64)
    assert need >= 2 * 152 * 20 * 130 * 4
    assert size(1024, 5, 32, 8, 128, 1 << 19) == need                  # grows with neither B nor Lmax
    assert _attend(fn, B=0, q=0, ws=0) == b.SPECDEC_OK
    for bad in ({"D": 96}, {"n": 0}, {"n": 129}, {"Hq": 30}, {"Hq": 4}, {"H": 0}, {"B": -1}, {"Lmax": 4},
                {"Lmax": (1 << 30) + 1}, {"B": 1 << 20, "Lmax": 1 << 20}, {"Hq": 129 * 8},
                {"B": 1 << 25, "Lmax": 5}):
        assert _attend(fn, **bad) == b.SPECDEC_ERR_UNSUPPORTED, bad
        shape = dict(B=1, n=5, Hq=32, H=8, D=128, Lmax=64)
        shape.update(bad)
        assert size(*shape.values()) == 0, bad
    for bad in ({"q": 0}, {"kc": 0}, {"vc": 0}, {"lens": 0}, {"out": 0}, {"q": P + 8}, {"out": P + 2},
                {"lens": P + 2}, {"slopes": P + 1}, {"qs": 4095}, {"qs": 4088}, {"qs": 4100}, {"qs": 1 << 31},
                {"scale": float("nan")}, {"scale": 1e-35}, {"cap": -1.0}, {"cap": 1e-35}, {"cap": 1001.0},
                {"cap": float("inf")}, {"window": -1},
                {"parent": (0, 0, 0, 0, 0)}, {"parent": (-1, 1, 0, 0, 0)}, {"parent": (-1, 0, 0, 3, 0)},
                {"parent": (-1, 0, -1, 0, 0)}):
        assert _attend(fn, **bad) == b.SPECDEC_ERR_INVALID_ARG, bad
    if "kv8" in name:
        assert _attend(fn, sk=0) == b.SPECDEC_ERR_INVALID_ARG
        assert _attend(fn, sv=P + 2) == b.SPECDEC_ERR_INVALID_ARG
    for bad in ({"ws": 0}, {"ws": WS + 8}, {"nb": need - 1}):
        assert _attend(fn, **bad) == b.SPECDEC_ERR_WORKSPACE, bad


def test_python_refuses_cpu_tensors():
    import target_model_verify_gb300 as tv
    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    codes, scales = x.to(torch.float8_e4m3fn), torch.ones(1, 4, 1)
    one = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(TypeError):
        tv.append_kv8(x, x, codes, codes, scales, scales, one)
    with pytest.raises(TypeError):
        tv.verify_attention_kv8(x, codes, codes, scales, scales, one)
    with pytest.raises(TypeError):
        tv.verify_attention_masked(x, x, x, one)
