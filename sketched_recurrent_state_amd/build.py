"""Build libsketchssm.so in-tree with hipcc for gfx950.

    python sketched_recurrent_state_amd/build.py [-j JOBS] [--save-temps]

Each HIP source compiles to its own object under ``_build/`` (in parallel),
then hipcc links the shared library next to this file.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libsketchssm.so")
SOURCES = ["abi.hip", "update_refresh.hip", "update_refresh_mamba2.hip", "update_refresh_gdn.hip",
           "update_refresh_kda.hip", "decode.hip", "sketch_decode_mamba2.hip",
           "sketch_decode_gdn.hip", "sketch_decode_kda.hip", "decode_step_mamba2.hip",
           "decode_step_gdn.hip", "decode_step_kda.hip", "append.hip", "recurrent.hip",
           "fit_basis.hip", "stream_probe.hip", "plan.hip", "scan_mamba2.hip", "scan_gdn.hip",
           "scan_kda.hip"]
ARCH = "gfx950"

HIPCC = os.environ.get("HIPCC", shutil.which("hipcc") or "/opt/rocm/bin/hipcc")

FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-Wall",
    # packed fp32 (v_pk_*_f32) stays off in every kernel
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # the scan asks for registers of two waves a SIMD also where LDS holds fewer (fp32, KDA):
    # with all registers the fp32 passes were 2 to 5 % slower
    "-Wno-pass-failed",
    "-I", INCLUDE, "-I", CSRC,
]


def _compile(src: str, save_temps: bool) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    if save_temps:
        cmd += ["-save-temps=obj"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    noise = "is not a recognized feature for this target"
    err = "\n".join(l for l in r.stderr.splitlines() if noise not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{err}")
    if err.strip():
        sys.stderr.write(err + "\n")
    return obj


def build(jobs: int = 0, save_temps: bool = False, verbose: bool = True) -> str:
    jobs = jobs or min(8, os.cpu_count() or 1)
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=max(1, jobs)) as ex:
        objs = list(ex.map(lambda s: _compile(s, save_temps), SOURCES))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}")
    return LIB


def main() -> None:
    ap = argparse.ArgumentParser()
    ap.add_argument("-j", "--jobs", type=int, default=min(8, os.cpu_count() or 1))
    ap.add_argument("--save-temps", action="store_true")
    a = ap.parse_args()
    build(a.jobs, a.save_temps)


if __name__ == "__main__":
    main()
