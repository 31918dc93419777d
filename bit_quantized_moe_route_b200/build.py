"""Build the layer's shared library (libmoe_lowbit.so) in-tree for sm_100a.

Usage: ``python -m bit_quantized_moe_route_b200.build [--force]``.
"""
from __future__ import annotations

import glob
import os
import re
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libmoe_lowbit.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC,-O2"]
OBJDIR = os.path.join(PKG, "_build")


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def inputs():
    return sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + sorted(
        glob.glob(os.path.join(CSRC, "*.inl"))) + sorted(glob.glob(os.path.join(CSRC, "*.h"))) + [os.path.join(ROOT, "include", "moe_lowbit.h")]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in inputs())


def launch_registers(src: str):
    """Registers per thread that the grouped kernel of `src` counts on when it starts (its warps share them out), or
    None: another source, or a kernel that leaves them as they are."""
    if not os.path.basename(src).startswith("gu_"):
        return None
    with open(src) as f:
        form = dict(re.findall(r"#define GU_(\w+) (\w+)", f.read()))
    with open(os.path.join(CSRC, "grouped_umma.cuh")) as f:
        regs = dict(re.findall(r"\b(kGuRegs|kGuAnyRegs) = (\d+)", f.read()))
    if form["ANY"] == "true":
        return int(regs["kGuAnyRegs"])
    return int(regs["kGuRegs"]) if form["MT"] != "1" or form["CHAIN"] != "0" else None


def check_registers(src: str, ptxas_log: str) -> None:
    """Raise unless ptxas gave the one kernel of `src` the registers it counts on (in the launch's units of 8)."""
    want = launch_registers(src)
    if want is None:
        return
    used = [int(n) for n in re.findall(r"Used (\d+) registers", ptxas_log)]
    if [-(-n // 8) * 8 for n in used] != [want]:
        raise RuntimeError(f"{os.path.basename(src)}: compiled to {used} registers, its warps share out {want} each")


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(OBJDIR, os.path.basename(src) + ".o")
    cmd = [nvcc(), *ARCH, *FLAGS, "-Xptxas", "-v", "-I", os.path.join(ROOT, "include"), "-c", "-o", obj, src]
    if verbose:
        print(" ".join(cmd), flush=True)
    run = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if run.returncode:
        raise RuntimeError(f"nvcc failed on {src}:\n{run.stdout}")
    for line in run.stdout.splitlines():
        if "warning" in line:
            print(line, flush=True)
    try:
        check_registers(src, run.stdout)
    except RuntimeError:
        os.remove(obj)
        raise
    return obj


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every translation unit (in parallel) and link libmoe_lowbit.so."""
    if not force and up_to_date():
        return LIB
    from concurrent.futures import ThreadPoolExecutor
    os.makedirs(OBJDIR, exist_ok=True)
    srcs = sources()
    headers = [p for p in inputs() if not p.endswith(".cu")]
    newest_header = max(os.path.getmtime(p) for p in headers)
    todo = []
    for src in srcs:
        obj = os.path.join(OBJDIR, os.path.basename(src) + ".o")
        if force or not os.path.exists(obj) or os.path.getmtime(obj) < max(os.path.getmtime(src), newest_header):
            todo.append(src)
    workers = max(1, min(len(todo), os.cpu_count() or 1))
    with ThreadPoolExecutor(max_workers=workers) as ex:
        list(ex.map(lambda s_: _compile(s_, verbose), todo))
    objs = [os.path.join(OBJDIR, os.path.basename(s_) + ".o") for s_ in srcs]
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
