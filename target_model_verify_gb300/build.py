"""Builds libspecdec_verify.so (the C-ABI library) in-tree for sm_103a.

    python -m target_model_verify_gb300.build [--force] [--verbose]

Each .cu file under csrc/ compiles to an object in parallel with nvcc; the
objects link into target_model_verify_gb300/_lib/libspecdec_verify.so with
the CUDA runtime linked statically. csrc/native.cpp (argument marshalling
against PyTorch's headers) compiles alongside with the host compiler into
_lib/_native.so; where that fails (no PyTorch, none of its headers), the
library is built all the same and only the operators that need the module
raise. Each is rebuilt only when one of its sources or headers is newer, the
module also for another PyTorch or Python.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_lib")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_NAME = "libspecdec_verify.so"
LIB_PATH = os.path.join(OUT_DIR, LIB_NAME)
NATIVE_SRC = os.path.join(CSRC, "native.cpp")
NATIVE_PATH = os.path.join(OUT_DIR, "_native.so")

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(INCLUDE, "*.h")))


def _newer_than(path, files) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(f) <= os.path.getmtime(path) for f in files)


def _library_up_to_date() -> bool:
    return _newer_than(LIB_PATH, _sources() + _headers() + [__file__])


def _torch_id() -> str:
    """What the module is built against: the Python, and PyTorch's version and place."""
    import importlib.metadata
    import importlib.util
    try:
        spec, version = importlib.util.find_spec("torch"), importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        spec, version = None, "none"
    return f"{sys.implementation.cache_tag} torch {version} {spec.origin if spec else ''}\n"


def _native_up_to_date() -> bool:
    if not _newer_than(NATIVE_PATH, glob.glob(os.path.join(INCLUDE, "*.h")) + [NATIVE_SRC, __file__]):
        return False
    try:
        with open(os.path.join(BUILD_DIR, "native.for"), encoding="utf-8") as f:
            return f.read() == _torch_id()
    except OSError:
        return False


def up_to_date() -> bool:
    return _library_up_to_date() and _native_up_to_date()


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc(), *ARCH_FLAGS, *NVCC_FLAGS, "-c", src, "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{res.stderr}")
    if verbose and res.stderr:
        sys.stderr.write(res.stderr)
    return obj


def _compile_native() -> str:
    """The host-side object of the Python module (g++ against PyTorch's headers)."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    obj = os.path.join(BUILD_DIR, "native.o")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    incs = [INCLUDE, *cpp_extension.include_paths(), sysconfig.get_paths()["include"], cuda]
    cmd = ["g++", "-O1", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(x for i in incs for x in ("-isystem" if "torch" in i else "-I", i)),
           "-c", NATIVE_SRC, "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed on native.cpp:\n{res.stderr}")
    return obj


def _link_native(obj: str) -> None:
    from torch.utils import cpp_extension
    tmp = NATIVE_PATH + ".tmp"
    libs = [x for p in cpp_extension.library_paths() for x in (f"-L{p}", f"-Wl,-rpath,{p}")]
    cmd = ["g++", "-shared", "-o", tmp, obj, f"-L{OUT_DIR}", f"-l:{LIB_NAME}", "-Wl,-rpath,$ORIGIN", *libs,
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"linking _native.so failed:\n{res.stderr}")
    with open(os.path.join(BUILD_DIR, "native.for"), "w", encoding="utf-8") as f:
        f.write(_torch_id())
    os.replace(tmp, NATIVE_PATH)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link the library, and the Python module where that can be built; returns the
    library's path."""
    need_lib, need_native = force or not _library_up_to_date(), force or not _native_up_to_date()
    if not need_lib and not need_native:
        return LIB_PATH
    os.makedirs(OUT_DIR, exist_ok=True)
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs = _sources() if need_lib else []
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        native = ex.submit(_compile_native) if need_native else None
        objs = list(ex.map(lambda s: _compile(s, verbose), srcs))
    if need_lib:
        tmp = LIB_PATH + ".tmp"
        cmd = [nvcc(), *ARCH_FLAGS, "-shared", "-o", tmp, *objs]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stderr}")
        os.replace(tmp, LIB_PATH)
    if need_native:
        try:
            _link_native(native.result())
        except (ImportError, RuntimeError, OSError) as e:
            if os.path.exists(NATIVE_PATH):                # of older sources
                os.remove(NATIVE_PATH)
            sys.stderr.write(f"warning: _native.so was not built, append_kv8() and the cache attention "
                             f"will raise from Python:\n{e}\n")
    return LIB_PATH


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true", help="print ptxas resource usage")
    args = ap.parse_args(argv)
    print(build(force=args.force, verbose=args.verbose))


if __name__ == "__main__":
    main()
