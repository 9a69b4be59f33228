"""The build script: what is built where parts cannot be, and what makes a part stale (CPU)."""
import os
import subprocess

import pytest

from target_model_verify_gb300 import build as libbuild


@pytest.fixture
def sandbox(tmp_path, monkeypatch):
    """The build's outputs in a folder of their own, its compilers replaced by ones that write the file
    they are asked for; `fail` names programs that report an error instead."""
    monkeypatch.setattr(libbuild, "OUT_DIR", str(tmp_path / "_lib"))
    monkeypatch.setattr(libbuild, "BUILD_DIR", str(tmp_path / "_build"))
    monkeypatch.setattr(libbuild, "LIB_PATH", str(tmp_path / "_lib" / "lib.so"))
    monkeypatch.setattr(libbuild, "NATIVE_PATH", str(tmp_path / "_lib" / "_native.so"))
    monkeypatch.setattr(libbuild, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    ran, fail = [], set()

    def run(cmd, **_):
        name = os.path.basename(cmd[0])
        ran.append((name, [c for c in cmd if c.endswith((".cu", ".cpp"))]))
        if name in fail:
            return subprocess.CompletedProcess(cmd, 1, "", "fatal error: ATen/ATen.h: No such file or directory")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("x")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(subprocess, "run", run)
    return ran, fail


def test_the_library_is_built_without_pytorchs_headers(sandbox, capsys):
    ran, fail = sandbox
    fail.add("g++")
    assert libbuild.build() == libbuild.LIB_PATH
    assert os.path.exists(libbuild.LIB_PATH) and not os.path.exists(libbuild.NATIVE_PATH)
    assert "ATen.h" in capsys.readouterr().err
    assert not libbuild.up_to_date()
    # the next time only the missing part is tried
    del ran[:]
    fail.clear()
    libbuild.build()
    assert os.path.exists(libbuild.NATIVE_PATH) and {name for name, _ in ran} == {"g++"}
    assert libbuild.up_to_date()
    del ran[:]
    libbuild.build()
    assert not ran


def test_a_module_of_older_sources_is_not_left(sandbox):
    ran, fail = sandbox
    libbuild.build()
    assert os.path.exists(libbuild.NATIVE_PATH)
    fail.add("g++")
    libbuild.build(force=True)
    assert os.path.exists(libbuild.LIB_PATH) and not os.path.exists(libbuild.NATIVE_PATH)


def test_a_failing_kernel_fails_the_build(sandbox):
    _, fail = sandbox
    fail.add("nvcc")
    with pytest.raises(RuntimeError):
        libbuild.build()


def test_another_pytorch_makes_the_module_stale(sandbox, monkeypatch):
    ran, _ = sandbox
    libbuild.build()
    assert libbuild.up_to_date()
    monkeypatch.setattr(libbuild, "_torch_id", lambda: "cpython-399 torch 9.9 elsewhere\n", raising=False)
    assert not libbuild.up_to_date()
    del ran[:]
    libbuild.build()
    assert {name for name, _ in ran} == {"g++"}                     # the module alone
    assert libbuild.up_to_date()


def test_the_module_names_the_pytorch_it_is_for():
    import torch
    assert torch.__version__.split("+")[0] in libbuild._torch_id()
    assert os.path.dirname(torch.__file__) in libbuild._torch_id()
