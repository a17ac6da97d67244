"""Build libadaspark.so in-tree with nvcc for sm_100a, and the Python binding of
the generation calls, _calls.so, with the host compiler (no GPU needed).

    python -m ffn_long_video_b200._build [-v]

Every .cu / .cpp under csrc/ is compiled separately (in parallel) into _build/
and linked into ffn_long_video_b200/libadaspark.so.  The CUDA runtime is linked
statically; the driver API is reached through cudaGetDriverEntryPoint.
binding/calls.cpp is compiled against the installed torch and linked to
libadaspark.so beside it. The library needs nvcc alone: where the binding cannot be
built (no torch, no Python headers), that is said on stderr, and only its calls
fail, when they are made.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libadaspark.so")
CALLS = os.path.join(PKG, "_calls.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC)
                  if f.endswith((".cu", ".cpp")))


def _compile(src: str, verbose: bool, ptxas_v: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    deps = [src] + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    deps.append(os.path.join(INCLUDE, "adaspark.h"))
    if (not ptxas_v and os.path.exists(obj)
            and os.path.getmtime(obj) >= max(os.path.getmtime(d) for d in deps)):
        return obj
    cmd = [_nvcc()] + ARCH + NVCC_FLAGS + (["-Xptxas", "-v"] if ptxas_v else []) + \
          ["-c", src, "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if ptxas_v or verbose:
        sys.stderr.write(r.stderr)
    return obj


def build(verbose: bool = False, ptxas_v: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose, ptxas_v), srcs))
    newest = max(os.path.getmtime(o) for o in objs)
    if not os.path.exists(LIB) or os.path.getmtime(LIB) < newest:
        cmd = [_nvcc()] + ARCH + ["-shared", "-o", LIB] + objs + ["-lpthread", "-ldl", "-lrt"]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    try:
        build_calls(verbose)
    except (ImportError, OSError, RuntimeError) as e:
        print(f"{os.path.basename(CALLS)}, the binding of the generation calls, was not built: {e}",
              file=sys.stderr)
    return LIB


def build_calls(verbose: bool = False) -> str:
    """_calls.so: the binding of the generation calls (needs libadaspark.so). Where it
    has to be built and cannot be, none is left behind."""
    import sysconfig

    import torch
    src = os.path.join(PKG, "binding", "calls.cpp")
    troot = os.path.dirname(os.path.abspath(torch.__file__))
    stamp = os.path.join(BUILD, "calls.torch")   # the torch and Python it was compiled against
    now = f"{torch.__version__} {sys.implementation.cache_tag}"
    said = open(stamp).read() if os.path.exists(stamp) else ""
    newest = max(os.path.getmtime(p) for p in (src, os.path.join(INCLUDE, "adaspark.h")))
    if os.path.exists(CALLS) and os.path.getmtime(CALLS) >= newest and said == now:
        return CALLS
    if os.path.exists(CALLS):
        os.remove(CALLS)
    tlib = os.path.join(troot, "lib")
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE, "-I", sysconfig.get_paths()["include"],
           "-I", os.path.join(troot, "include"),
           "-I", os.path.join(troot, "include", "torch", "csrc", "api", "include"),
           "-I", os.path.join(cuda, "include"), src, "-o", CALLS, "-L", PKG, "-l:libadaspark.so",
           "-L", tlib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python",
           "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"building _calls.so failed:\n{r.stdout}\n{r.stderr}")
    with open(stamp, "w") as f:
        f.write(now)
    return CALLS


if __name__ == "__main__":
    build(verbose="-v" in sys.argv, ptxas_v="--ptxas" in sys.argv)
    print(LIB)
