"""Build ``libpsa.so`` (the C-ABI library) in-tree with nvcc for sm_100a.

Usage: ``python -m block_sparse_attention_psa_b200.build [--ptxas-v]``.
Each ``csrc/*.cu`` is compiled to an object under ``_build/`` (in parallel,
skipped when up to date) and linked into ``libpsa.so`` next to this file.
``csrc/call.cpp`` (the binding's serving calls) becomes ``_call.so`` beside it.
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
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libpsa.so")
CALL = os.path.join(PKG, "_call.so")
CALL_STAMP = os.path.join(BUILD, "call.built_for")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _deps() -> list[str]:
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        [os.path.join(INCLUDE, "psa.h")]


def _compile(src: str, ptxas_v: bool) -> tuple[str, str]:
    obj = os.path.join(BUILD, os.path.basename(src).replace(".cu", ".o"))
    newest_dep = max(os.path.getmtime(p) for p in _deps() + [src])
    if os.path.exists(obj) and os.path.getmtime(obj) >= newest_dep and not ptxas_v:
        return obj, ""
    cmd = [_nvcc(), *ARCH, *FLAGS, "-c", src, "-o", obj]
    if ptxas_v:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr


def built_for() -> str:
    """The PyTorch and Python of this process, whose layouts ``_call.so`` has compiled in."""
    import torch

    return f"torch {torch.__version__} {torch.version.git_version} {sys.implementation.cache_tag}"


def _call_is_current(sources) -> bool:
    try:
        with open(CALL_STAMP) as f:
            return f.read() == built_for() and os.path.getmtime(CALL) >= max(os.path.getmtime(p) for p in sources)
    except OSError:
        return False


def _build_call() -> str:
    """The native form of the binding's serving calls, against the PyTorch and
    Python it is used with (others build it anew)."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension as ext

    src = os.path.join(CSRC, "call.cpp")
    if _call_is_current((src, os.path.join(INCLUDE, "psa.h"), torch.__file__)):
        return CALL
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    inc = [INCLUDE, *ext.include_paths(), os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = f"{CALL}.{os.getpid()}"   # a process that has the old one mapped keeps it
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", f'-DPSA_BUILT_FOR="{built_for()}"',
           *(f"-isystem{p}" for p in inc), src, "-o", tmp, "-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {src}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALL)
    with open(CALL_STAMP, "w") as f:
        f.write(built_for())
    return CALL


def build(ptxas_v: bool = False, verbose: bool = False) -> str:
    """Compile every CUDA source for sm_100a and link ``libpsa.so``, and the
    binding's ``_call.so``.  The library needs nvcc alone; where ``_call.so``
    cannot be built (no PyTorch, no Python headers, no g++) the binding does
    without it, and this says why on stderr."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs) + 1)) as ex:
        call = ex.submit(_build_call)
        results = list(ex.map(lambda s: _compile(s, ptxas_v), srcs))
        try:
            call.result()
        except Exception as e:
            if os.path.exists(CALL):   # of other sources: its calls may not be the library's
                os.remove(CALL)
            sys.stderr.write(f"_call.so is not built (the serving calls take longer on the host): {e}\n")
    objs = [o for o, _ in results]
    if verbose or ptxas_v:
        for _, log in results:
            if log:
                sys.stderr.write(log)
    newest_obj = max(os.path.getmtime(o) for o in objs)
    if not os.path.exists(LIB) or os.path.getmtime(LIB) < newest_obj:
        cmd = [_nvcc(), *ARCH, "-shared", "-o", LIB, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--ptxas-v", action="store_true", help="print register / spill / smem usage")
    args = ap.parse_args()
    print(build(ptxas_v=args.ptxas_v, verbose=True))
