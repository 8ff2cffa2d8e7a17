"""Build libvsa.so (the sm_103a CUDA library) in-tree with nvcc.

Every translation unit in csrc/ is compiled in parallel for sm_103a only
(-gencode arch=compute_103a,code=sm_103a) and linked into csrc/../_build/libvsa.so with the CUDA
runtime linked statically; the driver API (tensor-map encoding) is reached through
cudaGetDriverEntryPointByVersion, so the library loads on machines without a GPU driver.
"""
import concurrent.futures
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libvsa.so")
SOURCES = ["api.cu", "invert.cu", "prepost.cu", "tmap.cu", "bwd_main.cu", "fwd_main.cu",
           "noalloc.cu", "layer_api.cu", "norm_rope.cu", "cross_fwd.cu", "cross_token.cu",
           "cross_bwd.cu", "block_api.cu", "gate_norm.cu", "linear.cu",
           "gemm.cu", "gemm_small.cu", "linear_rows.cu"]
HEADERS = ["ptx.cuh", "queue.cuh", "vsa_internal.cuh", "layer_internal.cuh",
           "cross_common.cuh", "block_internal.cuh", "vec8.cuh", "act.cuh",
           "gemm.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def _nvcc():
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build libvsa.so")
    return exe


def _inputs():
    files = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    files += [os.path.join(ROOT, "include", h) for h in ("vsa.h", "vsa_layer.h", "vsa_block.h")]
    return files


def up_to_date():
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build(force=False, verbose=False, ptxas_info=False):
    """Compile and link libvsa.so if any source changed.  Returns the library path."""
    if not force and not ptxas_info and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc] + ARCH + FLAGS + extra + ["-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed on %s:\n%s%s" % (src, r.stdout, r.stderr))
        if ptxas_info or verbose:
            sys.stdout.write(r.stderr)
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + ".%d.tmp" % os.getpid()
    cmd = [nvcc] + ARCH + ["-shared", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc link failed:\n%s%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas-info" in sys.argv)
    print(LIB)
