"""Build the HIP library libtmoe.so for gfx950 with hipcc (in-tree, no JIT cache)."""
from __future__ import annotations

import concurrent.futures
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OBJ = os.path.join(ROOT, "_build", "obj")
LIB = os.path.join(HERE, "libtmoe.so")
SOURCES = ["k_route_map.hip", "k_rowops.hip", "k_trellis_gemm.hip", "k_small_arm.hip", "k_router.hip", "k_mxfp4_quant.hip",
           "k_mxfp4_gemm.hip", "k_mxfp8_quant.hip", "k_norm.hip", "k_grouped_bf16.hip", "k_grouped_f16.hip",
           "k_grouped_mxfp8.hip", "tmoe_host.cpp", "tmoe_router_host.cpp", "tmoe_mxfp4_host.cpp", "tmoe_norm_host.cpp",
           "tmoe_grouped_host.cpp"]
HEADERS = ["tmoe_device.hpp", "tmoe_hadamard.hpp", "tmoe_internal.hpp", "tmoe_rowbody.hpp", "tmoe_routemap.hpp",
           "tmoe_router.hpp", "tmoe_mxfp4.hpp", "tmoe_mxfp8.hpp", "tmoe_norm.hpp", "tmoe_grouped.hpp", "tmoe_grouped_scales.hpp",
           "k_grouped.hpp"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "-x", "hip", "-std=c++20", "-O3", "-fPIC", "--offload-arch=gfx950",
    # no packed-fp32 instructions anywhere in device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-fno-gpu-rdc", "-Wall", "-Wno-unused-function",
    "-I", os.path.join(ROOT, "include"), "-I", CSRC,
]


# Per-source flags. The row kernels' MFMAs (the rotations of rows of 512 and 1024 values in the
# activation and the combine at large batches) keep their results in ordinary VGPRs: accumulation
# registers would cost those kernels occupancy and a copy of every result.
EXTRA = {"k_rowops.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"]}


def _compile(src: str, verbose: bool) -> str:
    out = os.path.join(OBJ, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *FLAGS, *EXTRA.get(src, []), "-c", os.path.join(CSRC, src), "-o", out]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    msgs = "\n".join(l for l in (r.stdout + r.stderr).splitlines()
                     if "packed-fp32-ops" not in l and "not a recognized feature" not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{msgs}")
    if msgs.strip() and verbose:
        print(msgs, file=sys.stderr)
    return out


def build(verbose: bool = False) -> str:
    os.makedirs(OBJ, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=4) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, "-shared", "-fPIC", "--offload-arch=gfx950", "-o", tmp, *objs]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
