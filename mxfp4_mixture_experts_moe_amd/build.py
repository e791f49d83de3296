"""Build libk3moe.so (HIP for gfx950) in-tree.

    python mxfp4_mixture_experts_moe_amd/build.py

Run it by path (or load it with importlib from its path): importing the
package itself loads the library, which must not be required to build it.

Every .hip source under csrc/ is compiled to an object with hipcc for gfx950
(in parallel), then linked into ``libk3moe.so`` next to this file.  hipcc
cross-compiles, so this runs on a machine without a GPU.
"""

from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG_DIR, "csrc")
BUILD_DIR = os.path.join(PKG_DIR, "_build")
LIB_NAME = "libk3moe.so"
LIB_PATH = os.path.join(PKG_DIR, LIB_NAME)
INCLUDE = os.path.join(os.path.dirname(PKG_DIR), "include")

SOURCES = ["abi.hip", "route.hip", "codec.hip", "group.hip", "ffn.hip", "ffn_big.hip", "ffn_stream.hip", "ffn_q4k.hip", "verify.hip", "cache.hip", "dense.hip",
           "quant.hip", "mxprod.hip", "layer.hip",
           "mx8.hip", "mx8prod.hip", "route_groups.hip", "verify_draft.hip"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-fno-gpu-flush-denormals-to-zero",  # the codec relies on exact fp32 subnormals
    # keep the compiler from forming packed-fp32 (v_pk_*_f32) instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
    f"-I{INCLUDE}",
]


# per-source additions: the Q4_K GEMM consumes every MFMA result in VALU
# arithmetic, so its accumulators stay in VGPRs (no AGPR copies); the few-token
# layer's change places every stage
EXTRA_FLAGS = {"ffn_q4k.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"], "layer.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"]}


def _compile(src: str) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *FLAGS, *EXTRA_FLAGS.get(src, []), "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj


def build(verbose: bool = True) -> str:
    """Compile every HIP source and link the shared library; returns its path."""
    if shutil.which(HIPCC) is None and not os.path.exists(HIPCC):
        raise RuntimeError(f"hipcc not found ({HIPCC})")
    os.makedirs(BUILD_DIR, exist_ok=True)
    jobs = min(len(SOURCES), int(os.environ.get("MAX_JOBS", "8")))
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB_PATH + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    if verbose:
        print(f"built {LIB_PATH}")
    return LIB_PATH


if __name__ == "__main__":
    try:
        build()
    except RuntimeError as e:
        print(e, file=sys.stderr)
        sys.exit(1)
