"""Build libna.so in-tree: every CUDA translation unit is compiled for sm_103a in parallel with nvcc
and linked into neighborhood_attention_fwd_gb300/_build/libna.so (git-ignored)."""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libna.so")
SOURCES = ["na_api.cu", "na_fma.cu", "na_tc.cu", "na_tc_f16.cu", "na_tc_sb3.cu", "na_unfused.cu",
           "na_rope.cu", "na_norm.cu", "na_winsoft.cu", "na_addnorm.cu", "na_glu.cu"]
SOURCES += [f"na_add_{way}_{t}.cu" for way in ("fwd", "bwd") for t in ("bf16", "f16", "f32")]
SOURCES += [f"na_glu_fma_{t}.cu" for t in ("bf16", "f16", "f32")]
SOURCES += [f"na_glu_{part}_{t}.cu" for part in ("fwd", "slopes", "grads") for t in ("bf16", "f16")]
SOURCES += [f"na_win_{form}_{way}_{t}.cu" for form in ("soft", "diff") for way in ("fwd", "bwd") for t in ("bf16", "f16", "f32")]
HEADERS = ["na_internal.h", "na_device.cuh", "na_tc_impl.cuh", "na_elem.cuh", "na_block.cuh",
           "na_win.h", "na_win_impl.cuh", "na_rows.cuh", "na_add.h", "na_add_impl.cuh", "na_machine.h",
           "na_glu_plan.h", "na_glu.h", "na_glu_tc.cuh", "na_glu_fma.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I" + os.path.join(ROOT, "include")]


def _nvcc() -> str:
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        raise RuntimeError("nvcc not found")
    return nvcc


def _stale(out: str, deps) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    hdrs = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(ROOT, "include", "na.h")]
    jobs = []
    objs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s] + hdrs):
            jobs.append([nvcc, *ARCH, *FLAGS, "-c", s, "-o", o])

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        if verbose:
            print(r.stdout + r.stderr)

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        list(ex.map(run, jobs))
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        run([nvcc, *ARCH, "-shared", "-o", tmp, *objs])
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
