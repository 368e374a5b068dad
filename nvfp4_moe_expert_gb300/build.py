"""Build libnvfp4moe.so (sm_103a) in-tree with nvcc: one object per .cu,
compiled in parallel, then linked into a shared library next to this file.

    python -m nvfp4_moe_expert_gb300.build [--force] [--verbose]
"""

import argparse
import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_NAME = "libnvfp4moe.so"
LIB_PATH = os.path.join(HERE, LIB_NAME)
SOURCES = ["quant.cu", "gemm.cu", "combine.cu", "router.cu", "api.cu", "route_noalloc.cu", "backward.cu", "route_topk.cu",
           "balance.cu",
           "balance_backward.cu",
           "mxfp4.cu", "linear.cu", "linear_pair.cu", "linear_quant.cu", "lora.cu", "lora_few_forward_bf16.cu",
           "lora_few_forward_f16.cu", "lora_few_backward.cu", "lora_grad.cu"] + [
    f"lora_many_{what}_to_{out}.cu" for what in ("forward_bf16", "forward_f16", "backward") for out in ("bf16", "f16", "f32")]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", BUILD_DIR]
SILU_GEN = os.path.join(HERE, "silu_table.py")
SILU_INC = os.path.join(BUILD_DIR, "silu_table.inc")


def _nvcc():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libnvfp4moe.so")


def _deps():
    return [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "nvfp4_moe.h"), SILU_GEN]


def _silu_table():
    """Generate the SiLU table initialiser gemm.cu compiles in (when missing or stale)."""
    if os.path.exists(SILU_INC) and os.path.getmtime(SILU_INC) >= os.path.getmtime(SILU_GEN):
        return
    from . import silu_table
    tmp = SILU_INC + ".tmp"
    silu_table.write_inc(tmp)
    os.replace(tmp, SILU_INC)


def up_to_date():
    if not os.path.exists(LIB_PATH):
        return False
    t = os.path.getmtime(LIB_PATH)
    return all(os.path.getmtime(p) <= t for p in _deps())


def build(force=False, verbose=False):
    """Compile and link; returns the library path."""
    if not force and up_to_date():
        return LIB_PATH
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    _silu_table()
    extra = ["-Xptxas", "-v"] if verbose else []

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        cmd = [nvcc] + NVCC_FLAGS + extra + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            sys.stderr.write(r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB_PATH + ".tmp"
    cmd = [nvcc] + ARCH + ["-shared", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose))
