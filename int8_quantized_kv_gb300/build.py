"""Builds libkvq8.so in-tree with nvcc for sm_103a (GB300).

Each .cu under csrc/ is compiled to an object in parallel, then linked into
int8_quantized_kv_gb300/_build/libkvq8.so; what ptxas says of its kernels
(registers, spills) is kept beside each object and checked where a kernel
depends on it.  Rebuilds only when a source, a header or this file is newer
than the library.  `python -m int8_quantized_kv_gb300.build`
does the same from a shell.
"""
from __future__ import annotations

import glob
import os
import re
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(BUILD_DIR, "libkvq8.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


# Kernels whose warpgroups trade registers (setmaxnreg) within what the launch holds, which is the count that the compiler
# gives them: (mangled name, registers per thread that the shares add up to, kLaunchRegs in tiles.cu).
TRADING = [(r"tile_kernelILb[01]ELi128E", 72)]


def check_registers(src: str, ptxas: str) -> None:
    """Raises where ptxas -v reports another register count for a kernel of TRADING than its shares add up to: it would be
    refused at its launch (a share above the launch's registers would wait for ever)."""
    for name, regs in re.findall(r"Compiling entry function '(\S+)'.*?Used (\d+) registers", ptxas, re.S):
        for pattern, want in TRADING:
            if re.search(pattern, name) and int(regs) != want:
                raise RuntimeError(f"{src}: {name} has {regs} registers per thread, its warpgroups' shares need {want}")


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: libkvq8 needs the CUDA toolkit to build")
    return cand


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    return [__file__] + sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))


def needs_build() -> bool:
    if not os.path.exists(LIB_PATH):
        return True
    t = os.path.getmtime(LIB_PATH)
    return any(os.path.getmtime(f) > t for f in _inputs())


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile libkvq8.so (sm_103a) if stale; return its path."""
    if not force and not needs_build():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-Xptxas", "-v", "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        said = r.stdout + r.stderr
        check_registers(os.path.basename(src), said)
        with open(obj[:-2] + ".ptxas", "w") as f:
            f.write(said)
        if ptxas_info:
            sys.stderr.write(said)
        elif verbose:
            sys.stderr.writelines(x for x in said.splitlines(True) if "ptxas info" not in x and "bytes stack frame" not in x)
        return obj

    srcs = sources()
    with ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 1))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
