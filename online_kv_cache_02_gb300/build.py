"""Compile libtq.so in-tree for sm_103a (GB300) with nvcc.

Every translation unit is compiled in parallel to an object under _build/,
then linked into _build/libtq.so.  No cmake, no torch extension machinery.
"""

import concurrent.futures as cf
import os
import shutil
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libtq.so")
SOURCES = ["tq_api.cu", "tq_quantize.cu", "tq_quantize_tc.cu", "tq_quantize_pipe.cu", "tq_decode.cu", "tq_decode_lut.cu", "tq_noalloc.cu", "tq_search.cu", "tq_search_tc.cu", "tq_causal_tc.cu",
           "tq_generic.cu", "tq_kv8_append.cu", "tq_kv8_rows.cu", "tq_kv8_tc.cu", "tq_kv8_rows_shared.cu", "tq_kv8_tc_shared.cu",
           "tq_kv8_shared.cu", "tq_read.cu", "tq_read_tc.cu", "tq_prompt.cu", "tq_prompt_tc.cu", "tq_prompt_parts.cu",
           "tq_host.cpp"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2", "--expt-relaxed-constexpr"]


def _nvcc():
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libtq.so")
    return path


def _compile(nvcc, src, extra):
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc] + ARCH + FLAGS + extra + ["-c", os.path.join(CSRC, src), "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{res.stdout}\n{res.stderr}")
    return obj, res.stderr


def build(verbose=False, extra=()):
    """Build (or rebuild) _build/libtq.so; returns its path."""
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(lambda s: _compile(nvcc, s, list(extra)), SOURCES))
    if verbose:
        for _, log in results:
            if log.strip():
                print(log)
    objs = [o for o, _ in results]
    tmp = LIB + ".tmp"
    cmd = [nvcc] + ARCH + ["-shared", "-o", tmp] + objs + ["-lcudart"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(verbose=True, extra=sys.argv[1:]))
