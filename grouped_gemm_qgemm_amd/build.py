"""Build libqgemm.so (all gfx950 HIP kernels + the C ABI) in-tree with hipcc.

    python -m grouped_gemm_qgemm_amd.build        # or __graft_entry__.build()

Every call recompiles. Objects go to _build/ next to this file, the shared
library to grouped_gemm_qgemm_amd/libqgemm.so.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT = os.path.join(PKG, "libqgemm.so")
BUILD = os.path.join(PKG, "_build")
ARCH = os.environ.get("QG_OFFLOAD_ARCH", "gfx950")

HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"

COMMON = [
    "-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
    "-I", os.path.join(ROOT, "include"), "-I", CSRC,
    # keep the compiler from emitting packed-fp32 VALU instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
]


# Per-source flags. The decode kernels (a few microseconds each) take their
# arguments preloaded into SGPRs by the dispatcher instead of loading them from
# the kernel-argument segment at the start of every wave (about 0.25 us per
# launch); the long kernels gain nothing measurable from it.
# The attention kernels for few rows call their repeat pass, which is hardly ever
# taken, out of line. With register allocation across calls, what the callee uses
# decides what is left for the caller's loop: the registers that hold its spilled
# scalars went to scratch memory there (drafts on e4m3 heads of 128: 106 -> 160 us).
SOURCE_FLAGS = {
    "w4_decode.hip": ["-mllvm", "-amdgpu-kernarg-preload-count=16"],
    "attention_rows.hip": ["-mllvm", "-enable-ipra=0"],
}


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.hip")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    lang = ["-x", "hip"] if src.endswith(".hip") else ["-x", "hip"]
    cmd = [HIPCC, *COMMON, *SOURCE_FLAGS.get(os.path.basename(src), []), *lang, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    # warnings, but for the host pass not knowing the target feature above
    said = [line for line in r.stderr.splitlines() if "packed-fp32-ops" not in line and not line.endswith("warning generated when compiling for host.")]
    if said:
        print("\n".join(said), file=sys.stderr)
    return obj


def build(verbose: bool = True, jobs: int | None = None) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()
    jobs = jobs or min(8, len(srcs), os.cpu_count() or 1)
    with cf.ThreadPoolExecutor(jobs) as ex:
        objs = list(ex.map(_compile, srcs))
    tmp = OUT + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, OUT)
    if verbose:
        print(f"built {OUT} from {len(srcs)} sources")
    return OUT


if __name__ == "__main__":
    build()
    sys.exit(0)
