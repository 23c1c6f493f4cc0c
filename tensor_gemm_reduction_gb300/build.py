"""Build the CUDA library in-tree: ``tensor_gemm_reduction_gb300/_lib/libgsr.so``.

Each translation unit is compiled for sm_103a only (one ``-gencode``), in
parallel, and linked against the static CUDA runtime, so the library loads on a
machine without a GPU (the C-ABI tests check its exports there) and needs only
the driver on a GPU machine.

    python -m tensor_gemm_reduction_gb300.build [--force] [--verbose-ptxas]
"""
from __future__ import annotations

import argparse
import contextlib
import fcntl
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_lib")
LIB = os.path.join(OUT_DIR, "libgsr.so")
SOURCES = ["gsr_kernel.cu", "gsr_small.cu", "gsr_pack.cu", "gsr_api.cu", "gsr_routed.cu",
           "gsr_lowrank.cu", "gsr_route.cu", "gsr_routed_api.cu", "gsr_fp8.cu", "gsr_quant.cu",
           "gsr_fp8_api.cu", "gsr_layer.cu"]
HEADERS = [os.path.join(CSRC, "gsr_params.h"), os.path.join(CSRC, "gsr_device.cuh"),
           os.path.join(CSRC, "gsr_host.h"), os.path.join(CSRC, "gsr_routed.h"),
           os.path.join(CSRC, "gsr_fp8.h"), os.path.join(CSRC, "gsr_layer.h"),
           os.path.join(INCLUDE, "gsr.h")]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA library cannot be built")


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, s) for s in SOURCES] + HEADERS
    return any(os.path.getmtime(d) > t for d in deps)


@contextlib.contextmanager
def _build_lock():
    """One build at a time per tree: processes that start together (one per
    rank) would otherwise write the same object files."""
    os.makedirs(OUT_DIR, exist_ok=True)
    with open(os.path.join(OUT_DIR, ".build.lock"), "w") as fh:
        fcntl.flock(fh, fcntl.LOCK_EX)
        try:
            yield
        finally:
            fcntl.flock(fh, fcntl.LOCK_UN)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    if not force and not _stale():
        return LIB
    with _build_lock():
        # Another process may have finished the same build while this one waited.
        if not force and not _stale():
            return LIB
        return _build(verbose_ptxas)


def _build(verbose_ptxas: bool) -> str:
    nvcc = _nvcc()
    common = [nvcc, *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
              "-I", INCLUDE, "-I", CSRC]
    if verbose_ptxas:
        common += ["-Xptxas", "-v"]

    def compile_one(src: str) -> str:
        obj = os.path.join(OUT_DIR, src.replace(".cu", ".o"))
        cmd = common + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose_ptxas and r.stderr:
            sys.stderr.write(r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = f"{LIB}.{os.getpid()}.tmp"
    cmd = [nvcc, *ARCH, "-shared", "-Xcompiler", "-fPIC", "-cudart", "static", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


def main() -> None:
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose-ptxas", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose_ptxas=a.verbose_ptxas))


if __name__ == "__main__":
    main()
