"""Build libpace.so (HIP kernels + C ABI) in-tree for gfx950 with hipcc.

    python bit_recurrent_state_amd/build.py        # (a script: importing the package
                                                   #  would load the library first)

Every source is compiled each call (objects go to _build/, the library next to this
file), in parallel.  Packed-FP32 instruction selection is switched off for all device
code; fp32 division and square root are correctly rounded.
"""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OBJ = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libpace.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

SOURCES = ["pace_host.cpp", "pace_decode.hip", "pace_prefill.hip", "pace_baseline.hip", "pace_calib.hip",
           "pace_cache.cpp", "pace_rotary.hip", "pace_kv.hip", "pace_attention.hip", "pace_attention_int8.hip",
           "pace_attention_int4.hip", "pace_attention_fp8.hip", "pace_draft.cpp", "pace_draft_step.hip",
           "pace_draft_commit.hip", "pace_draft_verify.hip", "pace_cache_move.hip"]
# measurement kernels (include/pace_measure.h), a library of their own
MEASURE_SOURCES = ["pace_measure.hip"]
MEASURE_LIB = os.path.join(HERE, "libpace_measure.so")

COMMON = [
    "-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
    "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # matrix-core results in ordinary VGPRs: no accumulator-register moves
    "-mllvm", "-amdgpu-mfma-vgpr-form",
    "-I" + os.path.join(ROOT, "include"),
]
# NaN / Inf inputs are undefined by pace.h: min / max need no NaN quieting there.  The attention
# layers' operators (pace_cache.h) and the verification of drafts have defined results for them.
FINITE_ONLY = ["-fno-honor-nans"]
HONOR_NANS = {"pace_cache.cpp", "pace_rotary.hip", "pace_kv.hip", "pace_attention.hip", "pace_attention_int8.hip",
              "pace_attention_int4.hip", "pace_attention_fp8.hip", "pace_draft.cpp", "pace_draft_verify.hip", "pace_cache_move.hip"}


def _compile(src: str) -> str:
    obj = os.path.join(OBJ, os.path.splitext(src)[0] + ".o")
    lang = ["-x", "hip"] if src.endswith(".hip") else []
    extra = [] if src in HONOR_NANS else FINITE_ONLY
    cmd = [HIPCC, *COMMON, *extra, *lang, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj


def _link(objs, lib):
    tmp = lib + ".tmp"
    cmd = [HIPCC, "-shared", "-fPIC", f"--offload-arch={ARCH}", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)


def build(verbose: bool = False) -> str:
    os.makedirs(OBJ, exist_ok=True)
    srcs = SOURCES + MEASURE_SOURCES
    with ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = dict(zip(srcs, ex.map(_compile, srcs)))
    _link([objs[s] for s in SOURCES], LIB)
    _link([objs[s] for s in MEASURE_SOURCES], MEASURE_LIB)
    if verbose:
        print("built", LIB, "and", MEASURE_LIB)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
