"""Builds libmx.so in-tree with nvcc for sm_100a (cross-compiles without a GPU),
and the torch binding's small extension module with g++.

    python -m fp8_quantization_mx_b200.build [--force] [--verbose]

Flags: -O3, -lineinfo, IEEE float semantics (no fast math, no flush-to-zero,
IEEE division and square root), static CUDA runtime so that the library loads
on a host without a GPU.
"""

from __future__ import annotations

import argparse
import hashlib
import os
import subprocess
import sys
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libmx.so")

SOURCES = ["mx_api.cu", "mx_kernels.cu", "mx_bat.cu", "mx_gemm.cu", "mx_api128.cu", "mx_quant128.cu",
           "mx_norm128.cu", "mx_gemm128.cu"]
HEADERS = ["mx_device.cuh", "mx_launch.h", "mx_stream.cuh", "mx_tc.cuh", "mx_tile128.cuh",
           "mx_gemm128.h", "mx_pdl.cuh", "mx_rowvec.h"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-ftz=false", "-prec-div=true", "-prec-sqrt=true",
              "-fmad=true", "-Xcompiler", "-fPIC,-O2", "-cudart", "static"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


STAMP = LIB + ".srchash"

# The C++ marshalling of the torch binding's 128-element calls: an extension
# module against the torch it will run with.
FAST = os.path.join(PKG, "_fast128.so")
FAST_SRC = os.path.join(CSRC, "mx_fast128.cpp")


def build_fast(force: bool = False) -> str:
    """Builds _fast128.so unless the one in place was built from this source,
    torch and Python."""
    import sysconfig

    import torch
    with open(FAST_SRC, "rb") as f:
        h = hashlib.sha256(f.read())
    h.update(f"{torch.__version__} {sys.version}".encode())
    want, stamp = h.hexdigest(), FAST + ".srchash"
    if not force and os.path.exists(FAST) and _stamp(stamp) == want:
        return FAST
    troot = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc())) if os.path.sep in nvcc() else "/usr/local/cuda"
    inc = [os.path.join(troot, "include"), os.path.join(troot, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    lib = os.path.join(troot, "lib")
    abi = int(getattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", True))
    subprocess.run(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={abi}",
                    *(f"-I{d}" for d in inc), FAST_SRC, "-o", FAST + ".tmp", f"-L{lib}",
                    "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10"], check=True)
    os.replace(FAST + ".tmp", FAST)
    with open(stamp + ".tmp", "w") as f:
        f.write(want + "\n")
    os.replace(stamp + ".tmp", stamp)
    return FAST


def source_hash(extra=None) -> str:
    """SHA-256 over every source, header and flag the library is built from."""
    h = hashlib.sha256()
    paths = [os.path.join(CSRC, s) for s in SOURCES + HEADERS] + [os.path.join(INCLUDE, "mx.h"),
                                                                   os.path.abspath(__file__)]
    for p in paths:
        h.update(os.path.basename(p).encode() + b"\0")
        with open(p, "rb") as f:
            h.update(f.read())
    h.update(" ".join(ARCH + NVCC_FLAGS + list(extra or [])).encode())
    return h.hexdigest()


def _stamp(path: str = STAMP) -> str:
    try:
        with open(path) as f:
            return f.read().strip()
    except OSError:
        return ""


def build(force: bool = False, verbose: bool = False, extra=None) -> str:
    """Builds libmx.so unless the one in place was built from these exact
    sources and flags (its recorded source hash matches); file times are not
    trusted, so a stale library is always rebuilt. The torch binding's
    extension module is kept up to date beside it; where it cannot be built,
    Python makes its calls."""
    lib = build_library(force, verbose, extra)
    try:
        build_fast(force)
    except (ImportError, OSError, subprocess.CalledProcessError) as e:
        if not isinstance(e, ImportError) and os.path.exists(FAST):
            os.remove(FAST)   # it may be of another source, torch or Python
        warnings.warn(f"{FAST} was not built, calls will take longer: {e}")
    return lib


def build_library(force: bool = False, verbose: bool = False, extra=None) -> str:
    """build() without the extension module."""
    want = source_hash(extra)
    if not force and not verbose and os.path.exists(LIB) and _stamp() == want:
        return LIB
    # one nvcc per source, in parallel, then one link
    base = [nvcc(), *ARCH, *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC]
    if verbose:
        base += ["-Xptxas", "-v"]
    base += list(extra or [])
    objs, procs = [], []
    for src in SOURCES:
        obj = os.path.join(CSRC, src.replace(".cu", ".o"))
        objs.append(obj)
        procs.append((src, subprocess.Popen(base + ["-c", os.path.join(CSRC, src), "-o", obj])))
    failed = [src for src, p in procs if p.wait() != 0]
    if failed:
        raise subprocess.CalledProcessError(1, f"nvcc {' '.join(failed)}")
    subprocess.run([nvcc(), *ARCH, "-shared", "-cudart", "static", *objs, "-o", LIB + ".tmp"],
                   check=True)
    for obj in objs:
        os.remove(obj)
    os.replace(LIB + ".tmp", LIB)
    with open(STAMP + ".tmp", "w") as f:
        f.write(want + "\n")
    os.replace(STAMP + ".tmp", STAMP)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    args = ap.parse_args()
    print(build(force=args.force or args.verbose, verbose=args.verbose), file=sys.stderr)
