"""Builds libfusedlinear.so (sm_103a) in-tree from csrc/*.cu and attention/*.cu.

Each translation unit is compiled by its own nvcc process in parallel, then
linked into one shared library next to this file.  Nothing is installed.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import re
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
ATTENTION = os.path.join(HERE, "attention")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libfusedlinear.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _flags():
    return ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
                   "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-I", ATTENTION]


def sources():
    return [os.path.join(d, f) for d in (CSRC, ATTENTION) for f in sorted(os.listdir(d)) if f.endswith(".cu")]


def _deps():
    return [os.path.join(d, f) for d in (CSRC, ATTENTION) for f in os.listdir(d)] + [
        os.path.join(ROOT, "include", "fused_linear.h")]


# Kernels whose warps share out the registers that they are launched with: with any other number than the one their
# source counts on they would not start.  Source file: (kernel, file and name of the constant).
REGISTERS = {f: ("attention_prefill_kernel", "prefill_attention_kernel.cuh", "kPreRegs")
             for f in ("k_attention_prefill.cu", "k_attention_prefill_window.cu", "k_attention_prefill_parts.cu")}


def check_registers(src: str, ptxas: str) -> None:
    """Raises unless ptxas (its -v output) gave every instance of the source's kernel the registers it counts on."""
    kernel, header, name = REGISTERS[os.path.basename(src)]
    with open(os.path.join(os.path.dirname(src), header), encoding="utf-8") as f:
        want = int(re.search(rf"\b{name} = (\d+)", f.read()).group(1))
    got = [int(used) for function, used in
           re.findall(r"Compiling entry function '(\w+)'.*?Used (\d+) registers", ptxas, re.S) if kernel in function]
    if not got or any(n != want for n in got):
        raise RuntimeError(f"{kernel}: compiled for {got} registers a thread, {name} counts on {want}")


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(d) <= t for d in _deps())


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    flags = _flags() + (extra or [])

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        counted = os.path.basename(src) in REGISTERS
        cmd = [nvcc] + flags + (["-Xptxas", "-v"] if counted else []) + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if counted:
            check_registers(src, r.stdout + r.stderr)
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=len(srcs)) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc] + ARCH + ["-shared", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    verbose = "-v" in sys.argv
    extra = ["-Xptxas", "-v"] if "--ptxas" in sys.argv else None
    print(build(force=True, verbose=verbose or extra is not None, extra=extra))
