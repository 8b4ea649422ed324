"""Build libgdn.so in-tree for sm_103a with nvcc (one translation unit per kernel file,
compiled in parallel, then linked), and the attention calls' marshalling module with gcc
(left out where Python's C headers are missing; attention.py does without it).
No torch, no cmake."""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libgdn.so")
MARSHAL = os.path.join(HERE, "_marshal.so")  # the attention calls' argument marshalling (CPython)
SOURCES = ["gdn_api.cu", "decode.cu", "chunk_f32.cu", "chunk_bf16.cu", "chunk_fused.cu", "chunk_tc.cu",
           "gdn_noalloc.cu", "block_io.cu", "rollback.cu", "split.cu", "decode_block.cu",
           "attn_api.cu", "attn_io.cu", "attn_tile.cu", "attn_step.cu",
           "attn_prefix.cu", "verify_tree.cu", "beam.cu", "beam_api.cu"]
HEADERS = ["common.cuh", "internal.h", "tc.cuh", "attn.h", "attn_tma.cuh",
           "attn_tile.cuh", "attn_step.cuh", "beam.h"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _flags(extra=()):
    return ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                   "-I", os.path.join(ROOT, "include"), "-I", CSRC] + list(extra)


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    """Compile (if stale) and link libgdn.so; returns its path."""
    os.makedirs(BUILD, exist_ok=True)
    hdrs = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(ROOT, "include", "gdn.h")]
    jobs = []
    objs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if force or ptxas_verbose or _stale(o, [s] + hdrs):
            extra = ["-Xptxas", "-v"] if ptxas_verbose else []
            jobs.append([nvcc()] + _flags(extra) + ["-c", s, "-o", o])

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
        return r.stdout + r.stderr

    if jobs:
        with concurrent.futures.ThreadPoolExecutor(max_workers=len(jobs)) as ex:
            for out in ex.map(run, jobs):
                if verbose or ptxas_verbose:
                    sys.stderr.write(out)
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + ".tmp%d" % os.getpid()
        run([nvcc()] + ARCH + ["-shared", "-o", tmp] + objs + ["-lcudart"])
        os.replace(tmp, LIB)
    src = os.path.join(CSRC, "marshal.c")
    python = sysconfig.get_paths()["include"]
    if not os.path.exists(os.path.join(python, "Python.h")):
        sys.stderr.write("no Python.h in %s: the attention calls' marshalling stays in Python\n" % python)
    elif force or _stale(MARSHAL, [src, os.path.join(ROOT, "include", "gdn.h")]):
        tmp = MARSHAL + ".tmp%d" % os.getpid()
        run(["gcc", "-O2", "-Wall", "-Wextra", "-fPIC", "-shared", "-I", python,
             "-I", os.path.join(ROOT, "include"), src, "-o", tmp])
        os.replace(tmp, MARSHAL)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True,
                ptxas_verbose="--ptxas-v" in sys.argv))
