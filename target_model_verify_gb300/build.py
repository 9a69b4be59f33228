"""Builds libspecdec_verify.so (the C-ABI library) in-tree for sm_103a.

    python -m target_model_verify_gb300.build [--force] [--verbose]

Each .cu file under csrc/ compiles to an object in parallel with nvcc; the
objects link into target_model_verify_gb300/_lib/libspecdec_verify.so with
the CUDA runtime linked statically. csrc/native.cpp (argument marshalling
against PyTorch's headers) compiles alongside with the host compiler into
_lib/_native.so. Everything is rebuilt only when a source or header is newer
than the built files.
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


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH) or not os.path.exists(NATIVE_PATH):
        return False
    t = min(os.path.getmtime(LIB_PATH), os.path.getmtime(NATIVE_PATH))
    return all(os.path.getmtime(f) <= t for f in _sources() + _headers() + [NATIVE_SRC, __file__])


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
    os.replace(tmp, NATIVE_PATH)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link the library; returns its path."""
    if not force and up_to_date():
        return LIB_PATH
    os.makedirs(OUT_DIR, exist_ok=True)
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        native = ex.submit(_compile_native)
        objs = list(ex.map(lambda s: _compile(s, verbose), srcs))
        native_obj = native.result()
    tmp = LIB_PATH + ".tmp"
    cmd = [nvcc(), *ARCH_FLAGS, "-shared", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stderr}")
    os.replace(tmp, LIB_PATH)
    _link_native(native_obj)
    return LIB_PATH


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true", help="print ptxas resource usage")
    args = ap.parse_args(argv)
    print(build(force=args.force, verbose=args.verbose))


if __name__ == "__main__":
    main()
