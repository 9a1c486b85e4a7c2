"""Builds libgqa.so (the CUDA kernels and the C ABI) in place with nvcc.

Every translation unit is compiled for sm_103a only, in parallel, then linked
into ``gqa_kv_cache_gb300/libgqa.so`` (CUDA runtime linked statically).
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libgqa.so")
BUILD = os.path.join(HERE, "_build")
SOURCES = ["gqa_api.cu", "gqa_simt.cu", "gqa_simt_f32_small.cu", "gqa_simt_f32_large.cu",
           "gqa_simt_bf16_small.cu", "gqa_simt_bf16_large.cu", "gqa_simt_f32_small_plain.cu",
           "gqa_simt_f32_large_plain.cu", "gqa_simt_bf16_small_plain.cu", "gqa_simt_bf16_large_plain.cu",
           "gqa_tc.cu", "gqa_tc_fine.cu", "gqa_tc_multi.cu", "gqa_unit.cu",
           "gqa_q4.cu", "gqa_scored.cu", *(f"gqa_scored_i8_{d}_{rows}{more}.cu" for d in (128, 64) for rows in ("few", "rows")
                                            for more in ("", "_more")), "gqa_scored_bf16_128.cu", "gqa_scored_bf16_64.cu",
           "gqa_rows.cu", "gqa_select.cu", "gqa_cache_api.cu",
           "gqa_rotate.cu", "gqa_evict.cu", "gqa_serve_api.cu",
           "gqa_validate.cu",
           "gqa_noalloc.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _flags():
    extra = os.environ.get("GQA_NVCC_FLAGS", "").split()   # e.g. -DGQA_TC_STAGES=4
    return ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                   "-I", INCLUDE, "-I", CSRC, "--expt-relaxed-constexpr", *extra]


def _stale(out, deps):
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    headers.append(os.path.join(INCLUDE, "gqa_decode.h"))
    objs, jobs = [], []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s, *headers, __file__]):
            cmd = [nvcc(), *_flags(), "-c", s, "-o", o]
            if ptxas_info:
                cmd += ["-Xptxas", "-v"]
            jobs.append(cmd)

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    if jobs:
        with cf.ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
            for cmd, r in ex.map(run, jobs):
                if verbose or ptxas_info or r.returncode:
                    sys.stderr.write(r.stdout + r.stderr)
                if r.returncode:
                    raise RuntimeError("nvcc failed: " + " ".join(cmd))
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        subprocess.check_call([nvcc(), *ARCH, "-shared", "-o", tmp, *objs])
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas-info" in sys.argv)
    print(LIB)
