"""In-tree build of libqw.so for sm_103a (GB300) with nvcc.

Each CUDA translation unit is compiled in parallel, then linked into
``decode_qwen3_decoder_gb300/_lib/libqw.so``. A stamp of the sources and flags skips the
build when nothing changed.
"""

from __future__ import annotations

import concurrent.futures as cf
import hashlib
import os
import re
import shutil
import subprocess
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIBDIR = os.path.join(PKG, "_lib")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(LIBDIR, "libqw.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O3",
                     "--expt-relaxed-constexpr", "-I", INCLUDE]
SOURCES = ["qw_runtime.cu", "k_small.cu", "k_attn.cu", "k_gemm.cu", "k_noalloc.cu", "k_sample.cu", "k_step.cu", "k_dec1.cu", "k_lmhead.cu",
           "k_kv8.cu", "k_kv8_attn.cu", "k_kv8_evict.cu", "k_mx.cu", "k_mx_gemm.cu"]
# Kernels that share their registers out by role at run time: the shares add up only if the compiler gives
# each thread exactly this many, and the library refuses to launch them otherwise.
REGISTERS = {"k_kv8_attn.cu": {"k_kv8_chunk": 128}}


def ptxas_log(src: str) -> str:
    """What ptxas -v said of a source with an entry in REGISTERS at the last build."""
    return os.path.join(BUILD, src.replace(".cu", ".ptxas"))


def check_registers(wanted: dict, log: str) -> None:
    """Raises unless every instance of the kernels in `wanted`, and one at least, has its number of registers in
    the output of ptxas -v."""
    used = re.findall(r"Compiling entry function '(\w+)'.*?Used (\d+) registers", log, re.S)
    for name, n in wanted.items():
        got = {int(r) for k, r in used if re.search(rf"\d{name}(?!_)", k)}
        if got != {n}:
            raise RuntimeError(f"{name} needs {n} registers a thread, the compiler gave {sorted(got)}")


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libqw")


def _stamp() -> str:
    h = hashlib.sha256()
    for f in sorted(os.listdir(CSRC)):
        h.update(f.encode())
        with open(os.path.join(CSRC, f), "rb") as fh:
            h.update(fh.read())
    with open(os.path.join(INCLUDE, "qw.h"), "rb") as fh:
        h.update(fh.read())
    h.update((" ".join(NVCC_FLAGS) + repr(REGISTERS)).encode())
    return h.hexdigest()


def build(verbose: bool = False, force: bool = False, extra_flags=()) -> str:
    """Compile libqw.so if the sources changed; returns its path."""
    os.makedirs(LIBDIR, exist_ok=True)
    os.makedirs(BUILD, exist_ok=True)
    stamp_file = os.path.join(BUILD, "libqw.stamp")
    stamp = _stamp() + "|" + " ".join(extra_flags)
    if not force and os.path.exists(LIB) and os.path.exists(stamp_file):
        if open(stamp_file).read() == stamp:
            return LIB
    nvcc = _nvcc()

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        verbose_ptxas = ["-Xptxas", "-v"] if src in REGISTERS else []
        cmd = [nvcc, *NVCC_FLAGS, *verbose_ptxas, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if src in REGISTERS:
            with open(ptxas_log(src), "w") as fh:
                fh.write(r.stdout + r.stderr)
            try:
                check_registers(REGISTERS[src], r.stdout + r.stderr)
            except RuntimeError as e:
                warnings.warn(f"{e}: calls that need it will be refused")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    with open(stamp_file, "w") as fh:
        fh.write(stamp)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True, force=True))
