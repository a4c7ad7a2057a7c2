"""Builds libgdr.so in-tree with nvcc for sm_103a.

Each CUDA translation unit is compiled in parallel, then linked into one
shared library whose only exported symbols are the gdr_* entry points of
include/gdr.h (the CUDA runtime is linked statically and kept private, so the
library binds to its own runtime even when PyTorch's is loaded too).
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import platform
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libgdr.so")
SOURCES = ["api.cu", "k_decode.cu", "k_short.cu", "k_chain.cu", "k_chain_fwd.cu", "k_chain_fwd_kv.cu", "k_chain_conv.cu", "k_chain_verify.cu",
           "k_chain_snap.cu", "k_fold.cu", "k_probe.cu",
           "layer/api_layer.cu", "layer/k_norm.cu", "layer/k_norm_odd.cu", "layer/k_norm_pairs.cu", "layer/k_la_step.cu", "layer/k_la_chunk.cu", "layer/k_la_small.cu",
           "layer/api_scan.cu", "layer/k_short_conv.cu", "layer/k_scan.cu", "layer/k_scan_bb.cu", "layer/k_scan_bf.cu", "layer/k_scan_ff.cu", "layer/k_scan_fx.cu", "layer/k_scan_step_bb.cu", "layer/k_scan_step_bf.cu",
           "layer/k_scan_step_ff.cu",
           "layer/k_accept.cu"]
HEADERS = ["gdr_internal.h", "gdr_device.cuh", "gdr_pipe.cuh", "gdr_state.cuh", "k_chain.cuh", "gdr.map",
           "layer/layer_internal.h", "layer/tc.cuh", "layer/k_norm.cuh", "layer/k_scan.cuh",
           "layer/k_scan_step.cuh", "layer/scan_device.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the GDR library needs the CUDA toolkit to build")


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(verbose: bool = False, ptxas_info: bool = False, force: bool = False) -> str:
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    # objects built on another host architecture (x86 vs aarch64) are never reused
    stamp = os.path.join(BUILD, "host.txt")
    host = platform.machine()
    if not os.path.exists(stamp) or open(stamp).read().strip() != host:
        force = True
        with open(stamp, "w") as f:
            f.write(host + "\n")
    hdrs = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(ROOT, "include", "gdr.h")]
    objs, jobs = [], []
    for s in SOURCES:
        src = os.path.join(CSRC, s)
        obj = os.path.join(BUILD, s.replace("/", "_").replace(".cu", ".o"))
        objs.append(obj)
        if force or _stale(obj, [src, *hdrs]):
            cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
            if ptxas_info:
                cmd += ["-Xptxas", "-v"]
            jobs.append(cmd)

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    if jobs:
        with cf.ThreadPoolExecutor(max_workers=len(jobs)) as ex:
            for cmd, r in ex.map(run, jobs):
                if verbose or ptxas_info or r.returncode:
                    sys.stderr.write(r.stdout + r.stderr)
                if r.returncode:
                    raise RuntimeError(f"nvcc failed: {' '.join(cmd)}")
    if force or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc, *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp, *objs,
               "-Xlinker", "--version-script=" + os.path.join(CSRC, "gdr.map")]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("link of libgdr.so failed")
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True, ptxas_info="-v" in sys.argv, force="-f" in sys.argv))
