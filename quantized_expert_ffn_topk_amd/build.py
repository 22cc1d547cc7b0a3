"""Builds libmoe.so (HIP kernels for gfx950 + the C ABI) and _calls.so (direct
calls of the operators from Python) in-tree.

    python -m quantized_expert_ffn_topk_amd.build

Objects go to _build/ at the repository root; the libraries land next to
this file.  Kernels are compiled with fp contraction off and packed-fp32 code
generation disabled.  _calls.so is left out where there is no Python.h or no
C++ compiler for it; those calls then go through ctypes.
"""
import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libmoe.so")
CALLS = os.path.join(PKG, "_calls.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CXX = os.environ.get("CXX", "g++")

HIP_SOURCES = ["kernels_router.hip", "kernels_gemv.hip", "kernels_bs1.hip", "kernels_gemm.hip",
               "kernels_mx.hip", "noalloc.hip", "kernels_probe.hip", "kernels_rows.hip",
               "kernels_linear.hip", "kernels_route.hip"]
CPP_SOURCES = ["api.cpp", "pack.cpp", "cache.cpp"]

COMMON = ["-O3", "-std=c++17", "-fPIC", "-ffp-contract=off", "-fno-fast-math", "-Wall",
          "-I" + os.path.join(ROOT, "include")]
DEVICE = ["-x", "hip", "--offload-arch=gfx950",
          "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
          "-mcumode"]


def _compile(src):
    path = os.path.join(CSRC, src)
    obj = os.path.join(BUILD, src + ".o")
    cmd = [HIPCC] + COMMON + DEVICE + ["-c", path, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    out = (r.stdout + r.stderr).strip()
    # the host pass does not know the packed-fp32 target feature; that warning is expected
    lines = [l for l in out.splitlines() if "packed-fp32-ops" not in l or "error" in l]
    if r.returncode != 0:
        raise RuntimeError("compile failed: %s\n%s" % (" ".join(cmd), "\n".join(lines)))
    return obj, "\n".join(lines)


def _link(cmd, lib, verbose):
    tmp = lib + ".tmp"
    r = subprocess.run(cmd + ["-o", tmp], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed: %s\n%s%s" % (" ".join(cmd), r.stdout, r.stderr))
    os.replace(tmp, lib)
    if verbose:
        print("built", lib, flush=True)


def build_calls(verbose=True):
    """Builds _calls.so; its path, or None where it cannot be built (then there is
    no file of an earlier build either)."""
    include = sysconfig.get_paths()["include"]
    missing = [what for what, there in (("Python.h in " + include, os.path.exists(os.path.join(include, "Python.h"))),
                                        (CXX, shutil.which(CXX.split()[0]))) if not there]
    if missing:
        if os.path.exists(CALLS):
            os.remove(CALLS)
        print("without %s: no _calls.so, the operators are called through ctypes" % " and ".join(missing), flush=True)
        return None
    _link(CXX.split() + ["-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-I" + os.path.join(ROOT, "include"),
                         "-I" + include, os.path.join(CSRC, "pycalls.cpp")], CALLS, verbose)
    return CALLS


def build(verbose=True, jobs=None):
    os.makedirs(BUILD, exist_ok=True)
    sources = HIP_SOURCES + CPP_SOURCES
    jobs = jobs or min(len(sources), os.cpu_count() or 4, 8)
    with cf.ThreadPoolExecutor(jobs) as ex:
        results = list(ex.map(_compile, sources))
    for (obj, msg), src in zip(results, sources):
        if verbose and msg:
            print("[%s]\n%s" % (src, msg), flush=True)
    _link([HIPCC, "-shared", "-fPIC", "--offload-arch=gfx950"] + [o for o, _ in results], LIB, verbose)
    build_calls(verbose)
    return LIB


if __name__ == "__main__":
    build()
    sys.exit(0)
