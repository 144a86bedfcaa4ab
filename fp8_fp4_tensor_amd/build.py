"""Build libfq.so (the HIP kernels and the C ABI of include/fq.h) for gfx950.

Every source is compiled with hipcc for gfx950 only, with
  -ffp-contract=off          no fused multiply-add: each product is rounded
                             once, as the quantization recipes define;
  no fast-math flags         fp32 division stays correctly rounded and
                             denormals are preserved (the gfx950 defaults);
  -packed-fp32-ops disabled  the compiler emits no packed fp32 VALU ops.
Objects go to fp8_fp4_tensor_amd/_build/, the library to
fp8_fp4_tensor_amd/libfq.so.
"""
import concurrent.futures
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libfq.so")
ARCH = "gfx950"

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-ffp-contract=off",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-Wall", "-Wno-unused-function", "-I", INCLUDE, "-I", CSRC]

SOURCES = ["api.cpp", "k_tensor.hip", "k_block.hip", "k_mx.hip", "k_mxfp4.hip", "k_nvfp4.hip", "k_dequant.hip", "k_requant.hip",
           "k_sr8.hip", "k_gemm.hip", "k_gemm_mx.hip", "k_gemm_mx_e4m3.hip",
           "k_gemm_mx_e5m2.hip", "k_gemm_mx_e2m1.hip", "k_norm.hip", "k_swiglu.hip", "k_kv.hip", "k_attn.hip", "noalloc.hip"]


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    lang = ["-x", "hip"] if src.endswith(".hip") else []
    cmd = [HIPCC, *FLAGS, *lang, "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    noise = "is not a recognized feature for this target"
    msg = "\n".join(l for l in (r.stdout + r.stderr).splitlines() if noise not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{msg}")
    if msg.strip() and verbose:
        print(msg, file=sys.stderr)
    return obj


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(SOURCES))) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
