"""Build the CUDA library (libbitlinear.so) in-tree with nvcc for sm_100a, and the
paged-cache calls' binding (_bind.<Python's ABI>.so) with the host compiler, where torch
and Python's headers are there: the library does without them.

    python -m bit_quantised_gemm_b200.build [--verbose]

Sources are compiled without fast-math: the quantisers rely on IEEE fp32
division and multiplication and on round-to-nearest-even conversions.
"""
from __future__ import annotations

import argparse
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libbitlinear.so")
BIND = os.path.join(PKG, "_bind" + sysconfig.get_config_var("EXT_SUFFIX"))
BIND_RECORD = os.path.join(PKG, "_build", "bind.txt")  # what BIND has been built with
SOURCES = ["api.cu", "quant.cu", "gemm.cu", "gemv.cu", "gemv_mma.cu", "gemv_dp4a.cu", "attn.cu", "paged.cu", "paged_attn.cu",
           "paged_front.cu", "peak.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale(out: str, deps: list[str]) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def build_binding(verbose: bool = False, force: bool = False) -> bool:
    """Build _bind where its source, torch or Python have changed; False if torch or a header is missing."""
    include = sysconfig.get_paths()["include"]
    torch = importlib.util.find_spec("torch")  # located, not imported
    missing = ([] if torch else ["torch"]) + ([] if os.path.exists(os.path.join(include, "Python.h")) else ["Python's headers"])
    if missing:
        print(f"the binding of the paged-cache calls is not built: no {' and no '.join(missing)}", file=sys.stderr)
        return False
    t = os.path.dirname(torch.origin)
    cuda = os.path.dirname(os.path.dirname(nvcc_path()))
    src = os.path.join(CSRC, "bind.cpp")
    # the system's g++, whose C++ runtime is torch's: a statically linked one breaks exceptions
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           "-I", os.path.join(t, "include"), "-I", os.path.join(t, "include", "torch", "csrc", "api", "include"),
           "-I", os.path.join(cuda, "include"), "-I", include, src, "-o", BIND,
           "-L", os.path.join(t, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    record = " ".join(cmd) + "\n" + open(os.path.join(t, "version.py")).read()
    known = open(BIND_RECORD).read() if os.path.exists(BIND_RECORD) else ""
    if not force and record == known and not _stale(BIND, [src, os.path.join(ROOT, "include", "bitlinear.h")]):
        return True
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    with open(BIND_RECORD, "w") as f:
        f.write(record)
    untagged = os.path.join(PKG, "_bind.so")  # of a build before the ABI was in the name
    if os.path.exists(untagged):
        os.remove(untagged)
    return True


def build(verbose: bool = False, force: bool = False) -> str:
    nvcc = nvcc_path()
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    headers.append(os.path.join(ROOT, "include", "bitlinear.h"))
    objdir = os.path.join(PKG, "_build")
    os.makedirs(objdir, exist_ok=True)
    objs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(objdir, src.replace(".cu", ".o"))
        objs.append(o)
        if not force and not _stale(o, [s] + headers):
            continue
        cmd = [nvcc, *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
               "-I", os.path.join(ROOT, "include"), "-c", s, "-o", o]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
    if force or _stale(LIB, objs):
        cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", LIB, *objs]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
    build_binding(verbose, force)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--force", action="store_true")
    a = ap.parse_args()
    print(build(verbose=a.verbose, force=a.force))
    sys.exit(0)
