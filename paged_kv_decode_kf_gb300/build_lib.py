"""Build the CUDA library in-tree: nvcc for sm_103a, one object per source
file compiled in parallel, linked into ``_lib/libkf.so``.

A stamp file next to the library holds a hash of the sources and flags, so
an unchanged tree is not rebuilt.
"""
from __future__ import annotations

import concurrent.futures as cf
import hashlib
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIBDIR = os.path.join(HERE, "_lib")
LIB = os.path.join(LIBDIR, "libkf.so")
SOURCES = ["kf_api.cu", "kf_append.cu", "kf_merge.cu", "kf_decode_simt.cu", "kf_decode_tc.cu",
           "kf_decode_tc_fp8.cu", "kf_decode_bal.cu", "kf_decode_bal_fp8.cu", "kf_multiquery.cu",
           "kf_multiquery_tc05.cu", "kf_multiquery_tc05w.cu", "kf_multiquery_tc05p.cu", "kf_static.cu",
           "kf_latent_api.cu", "kf_latent_append.cu", "kf_latent_tc05.cu",
           "kf_latent_expand.cu", "kf_latent_expanded.cu", "kf_accumulate.cu",
           "kf_accumulate_tc05.cu", "kf_evict.cu"]
HEADERS = [os.path.join(CSRC, "kf_internal.cuh"), os.path.join(CSRC, "kf_decode_tc.cuh"),
           os.path.join(CSRC, "kf_decode_bal.cuh"),
           os.path.join(CSRC, "kf_tc05.cuh"), os.path.join(CSRC, "kf_mq_tc05.cuh"),
           os.path.join(CSRC, "kf_latent.cuh"), os.path.join(CSRC, "kf_latent_expanded.cuh"),
           os.path.join(CSRC, "kf_runs.cuh"), os.path.join(CSRC, "kf_device.cuh"),
           os.path.join(CSRC, "kf_tc05_ops.cuh"), os.path.join(CSRC, "kf_evict.cuh"),
           os.path.join(ROOT, "include", "kf.h")]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I" + os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")


def _digest() -> str:
    h = hashlib.sha256()
    for f in [os.path.join(CSRC, s) for s in SOURCES] + HEADERS:
        with open(f, "rb") as fh:
            h.update(fh.read())
    h.update(" ".join(FLAGS).encode())
    h.update(os.uname().machine.encode())
    return h.hexdigest()


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(LIBDIR, exist_ok=True)
    stamp = LIB + ".stamp"
    digest = _digest()
    if not force and os.path.exists(LIB) and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read().strip() == digest:
                return LIB
    nvcc = _nvcc()
    objdir = os.path.join(LIBDIR, "obj")
    os.makedirs(objdir, exist_ok=True)

    def compile_one(src: str) -> str:
        obj = os.path.join(objdir, src.replace(".cu", ".o"))
        cmd = [nvcc] + FLAGS + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s%s" % (src, r.stdout, r.stderr))
        if verbose:
            sys.stdout.write(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + ".tmp%d" % os.getpid()
    r = subprocess.run([nvcc] + ARCH + ["-shared", "-o", tmp] + objs, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    with open(stamp, "w") as f:
        f.write(digest)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
