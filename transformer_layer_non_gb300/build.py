"""Build the C-ABI operator libraries for sm_103a with nvcc: ``libls_ops.so``
(the layer operators, ``csrc/``) and ``libls_vocab.so`` (the vocabulary
operators, ``csrc_vocab/``).

A library's translation units compile in parallel and link into
``transformer_layer_non_gb300/_build/``.  A rebuild happens only when a source
or header is newer than the library.  Usage::

    python -m transformer_layer_non_gb300.build [--force] [--verbose]
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libls_ops.so")
VOCAB_CSRC = os.path.join(PKG, "csrc_vocab")
VOCAB_LIB = os.path.join(BUILD, "libls_vocab.so")
# The benchmark's reference streaming kernel (not part of the operator library).
FLOOR_SRC = os.path.join(PKG, "floor", "stream_floor.cu")
FLOOR_LIB = os.path.join(BUILD, "libls_floor.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
                     "-Xcompiler", "-fPIC,-O3,-fvisibility=hidden", "-I", INCLUDE]


def _nvcc() -> str:
    for cand in [os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"]:
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libls_ops.so")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def vocab_sources():
    return sorted(glob.glob(os.path.join(VOCAB_CSRC, "*.cu")))


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(
        os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(INCLUDE, "*.h")) + [__file__]


def _vocab_headers():
    return _headers() + glob.glob(os.path.join(VOCAB_CSRC, "*.cuh")) + glob.glob(
        os.path.join(VOCAB_CSRC, "*.h"))


def _newer_than(lib: str, inputs) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(p) <= t for p in inputs)


def up_to_date() -> bool:
    return _newer_than(LIB, sources() + _headers())


def vocab_up_to_date() -> bool:
    return _newer_than(VOCAB_LIB, vocab_sources() + _vocab_headers())


def _compile_and_link(lib: str, srcs, obj_dir: str, verbose: bool, ptxas_verbose: bool) -> str:
    nvcc = _nvcc()
    os.makedirs(obj_dir, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_verbose else []

    def compile_one(src):
        obj = os.path.join(obj_dir, os.path.basename(src).replace(".cu", ".o"))
        cmd = [nvcc, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stdout + r.stderr

    with cf.ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        results = list(ex.map(compile_one, srcs))
    if verbose or ptxas_verbose:
        for obj, log in results:
            if log.strip():
                print(f"== {os.path.basename(obj)}\n{log}", file=sys.stderr)
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp] + [o for o, _ in results]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    """Compile and link the layer operators' library; returns its path."""
    if not force and up_to_date():
        return LIB
    return _compile_and_link(LIB, sources(), BUILD, verbose, ptxas_verbose)


def build_vocab(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    """Compile and link the vocabulary operators' library; returns its path."""
    if not force and vocab_up_to_date():
        return VOCAB_LIB
    return _compile_and_link(VOCAB_LIB, vocab_sources(), os.path.join(BUILD, "vocab"), verbose,
                             ptxas_verbose)


def build_floor(force: bool = False) -> str:
    """Compile the benchmark's reference streaming kernel into libls_floor.so."""
    if (not force and os.path.exists(FLOOR_LIB)
            and os.path.getmtime(FLOOR_LIB) >= max(os.path.getmtime(FLOOR_SRC),
                                                    os.path.getmtime(__file__))):
        return FLOOR_LIB
    os.makedirs(BUILD, exist_ok=True)
    tmp = FLOOR_LIB + f".tmp{os.getpid()}"
    cmd = [_nvcc(), *NVCC_FLAGS, "-shared", "-cudart", "static", "-o", tmp, FLOOR_SRC]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {FLOOR_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, FLOOR_LIB)
    return FLOOR_LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas", action="store_true", help="print -Xptxas -v register/spill report")
    a = ap.parse_args()
    print(build(force=a.force or a.ptxas, verbose=a.verbose, ptxas_verbose=a.ptxas))
    print(build_vocab(force=a.force or a.ptxas, verbose=a.verbose, ptxas_verbose=a.ptxas))
    print(build_floor(force=a.force))
