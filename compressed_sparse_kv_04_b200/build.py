"""Build libcsa.so in-tree for sm_100a (nvcc, one object per .cu, then link)
and _calls.so, the binding's native calls (g++, against torch's and Python's
headers).  libcsa.so needs nvcc alone: where torch or Python's headers are
missing, or _calls.so does not compile, it is built all the same.

    python -m compressed_sparse_kv_04_b200.build [--force]
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libcsa.so")
CALLS = os.path.join(PKG, "_calls.so")
CALLS_SRC = os.path.join(CSRC, "calls.cpp")
CALLS_TAG = os.path.join(BUILD, "calls.tag")  # what _calls.so was built for
HEADER = os.path.join(ROOT, "include", "csa.h")

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
         "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr", "-Xptxas", "-v"]


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _lib_deps():
    return [os.path.join(CSRC, f) for f in os.listdir(CSRC)
            if os.path.join(CSRC, f) != CALLS_SRC] + [HEADER]


def _newer(target, deps) -> bool:
    return os.path.exists(target) and all(
        os.path.getmtime(d) <= os.path.getmtime(target) for d in deps)


def can_build_calls() -> bool:
    """Whether what _calls.so compiles against is here."""
    return importlib.util.find_spec("torch") is not None and os.path.exists(
        os.path.join(sysconfig.get_paths()["include"], "Python.h"))


def _compile(src: str) -> tuple[str, str]:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [NVCC, *FLAGS, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
    with open(obj + ".ptxas.txt", "w") as f:
        f.write(r.stderr)
    return obj, r.stderr


def calls_tag() -> str:
    """What _calls.so depends on besides its sources: it is compiled against one
    torch's C++ types and one Python's."""
    import torch
    return (f"torch {torch.__version__}, C++11 ABI {int(torch._C._GLIBCXX_USE_CXX11_ABI)}, "
            f"Python {sysconfig.get_config_var('SOABI')}")


def _compile_calls() -> None:
    import torch
    t = os.path.dirname(torch.__file__)
    tmp = CALLS + ".tmp"
    tag = calls_tag()
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DCSA_CALLS_TAG="{tag}"',
           "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(t, "include"),
           "-I" + os.path.join(t, "include", "torch", "csrc", "api", "include"),
           "-I" + os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include"), CALLS_SRC,
           "-o", tmp, "-L" + os.path.join(t, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10",
           "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {CALLS_SRC}:\n{r.stderr}")
    os.replace(tmp, CALLS)
    with open(CALLS_TAG, "w") as f:
        f.write(tag)


def lib_up_to_date() -> bool:
    return _newer(LIB, _lib_deps())


def calls_up_to_date() -> bool:
    if not _newer(CALLS, [CALLS_SRC, HEADER]) or not os.path.exists(CALLS_TAG):
        return False
    with open(CALLS_TAG) as f:
        return f.read() == calls_tag()


def up_to_date() -> bool:
    return lib_up_to_date() and (not can_build_calls() or calls_up_to_date())


def _build_lib(verbose: bool) -> None:
    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        results = list(ex.map(_compile, srcs))
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    objs = [o for o, _ in results]
    tmp = LIB + ".tmp"
    cmd = [NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", tmp, *objs,
           "-lcudart"]
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        calls = None
        if not can_build_calls():
            sys.stderr.write("_calls.so is not built: it needs torch and Python's headers\n")
        elif force or not calls_up_to_date():
            calls = ex.submit(_compile_calls)
        if force or not lib_up_to_date():
            _build_lib(verbose)
        if calls is not None:
            calls.result()  # (libcsa.so is in place by now)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
