"""Builds libaq.so (the gfx950 HIP kernels and the C ABI) in-tree with hipcc, and the torch binding's module.

    python -m weight_only_bit_group_amd.build        # or build() from Python

Every call recompiles all sources.  Objects go to ``_build/`` at the repository
root; the shared library is written next to this file.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OBJ_DIR = os.path.join(ROOT, "_build")
LIB_PATH = os.path.join(HERE, "libaq.so")
# the ceiling microbenchmarks the benchmark runs beside the path (not part of the C ABI)
PROBE_SOURCE = os.path.join(CSRC, "probe", "ceiling.hip")
PROBE_PATH = os.path.join(HERE, "libaq_probe.so")

HIP_SOURCES = ("quant_pack.hip", "w4a16_gemv.hip", "decode_mfma.hip", "mfma_gemm.hip", "act_absmean.hip",
               "awq_search.hip", "fp4_gemv.hip", "fp4_quant.hip", "w8a16_gemv.hip", "mxfp4_quant.hip", "mxfp4_gemm.hip")
CPP_SOURCES = ("aq_api.cpp",)

# the torch binding's native calls, a CPython module linked against libaq.so beside it
TORCH_SOURCE = os.path.join(CSRC, "aq_torch.cpp")
TORCH_PATH = os.path.join(HERE, "_aq_torch.so")

COMMON_FLAGS = [
    "-O3", "-std=c++17", "-fPIC", "--offload-arch=gfx950",
    # Bit-exact quantization: IEEE division, no contraction into FMAs, no fast-math,
    # fp32 denormals preserved.
    "-ffp-contract=off", "-fno-fast-math", "-fno-gpu-flush-denormals-to-zero",
    # Keep the compiler from forming packed-fp32 VALU instructions.
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function", "-Wno-unused-variable",
    "-I" + os.path.join(ROOT, "include"),
]


def _hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm is required to build libaq)")


# Per-file extra flags: the GEMMs keep MFMA accumulators in VGPRs (the fp32
# group rescale operates on them with plain VALU FMAs).
FILE_FLAGS = {"mfma_gemm.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=true"]}


def _compile(src: str) -> str:
    obj = os.path.join(OBJ_DIR, os.path.basename(src) + ".o")
    cmd = [_hipcc(), *COMMON_FLAGS, *FILE_FLAGS.get(os.path.basename(src), []), "-c", os.path.join(CSRC, src), "-o", obj]
    proc = subprocess.run(cmd, capture_output=True, text=True)
    if proc.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{proc.stdout}\n{proc.stderr}")
    return obj


def _compile_torch() -> str:
    """The binding's host code, against torch's and Python's headers; no device code in it."""
    import torch

    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    obj = os.path.join(OBJ_DIR, os.path.basename(TORCH_SOURCE) + ".o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-Wall", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I" + os.path.join(ROOT, "include"),
           "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(os.path.dirname(os.path.dirname(_hipcc())), "include"),
           "-isystem", sysconfig.get_paths()["include"], "-c", TORCH_SOURCE, "-o", obj]
    proc = subprocess.run(cmd, capture_output=True, text=True)
    if proc.returncode != 0:
        raise RuntimeError(f"g++ failed for {TORCH_SOURCE}:\n{proc.stdout}\n{proc.stderr}")
    return obj


def _link_torch(obj: str) -> None:
    import torch

    tmp = TORCH_PATH + ".tmp"
    proc = subprocess.run(["g++", "-shared", "-fPIC", obj, "-L" + HERE, "-l:" + os.path.basename(LIB_PATH), "-Wl,-rpath,$ORIGIN",
                           "-L" + os.path.join(os.path.dirname(torch.__file__), "lib"), "-ltorch_python", "-ltorch_cpu",
                           "-lc10", "-lc10_hip", "-o", tmp], capture_output=True, text=True)
    if proc.returncode != 0:
        raise RuntimeError(f"link of the torch module failed:\n{proc.stdout}\n{proc.stderr}")
    os.replace(tmp, TORCH_PATH)


def build(verbose: bool = True) -> str:
    """Compile every source for gfx950, link libaq.so and the binding's module; returns the library path."""
    os.makedirs(OBJ_DIR, exist_ok=True)
    sources = list(HIP_SOURCES) + list(CPP_SOURCES)
    jobs = min(len(sources) + 2, max(1, min(8, os.cpu_count() or 1)))
    with ThreadPoolExecutor(max_workers=jobs) as pool:
        probe_obj = pool.submit(_compile, PROBE_SOURCE)
        torch_obj = pool.submit(_compile_torch)
        objs = list(pool.map(_compile, sources))
        probe_obj, torch_obj = probe_obj.result(), torch_obj.result()
    tmp = LIB_PATH + ".tmp"
    cmd = [_hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp]
    proc = subprocess.run(cmd, capture_output=True, text=True)
    if proc.returncode != 0:
        raise RuntimeError(f"link failed:\n{proc.stdout}\n{proc.stderr}")
    os.replace(tmp, LIB_PATH)
    _link_torch(torch_obj)
    tmp = PROBE_PATH + ".tmp"
    proc = subprocess.run([_hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC", probe_obj, "-o", tmp],
                          capture_output=True, text=True)
    if proc.returncode != 0:
        raise RuntimeError(f"probe link failed:\n{proc.stdout}\n{proc.stderr}")
    os.replace(tmp, PROBE_PATH)
    if verbose:
        print(f"built {LIB_PATH}, {TORCH_PATH} and {PROBE_PATH}")
    return LIB_PATH


if __name__ == "__main__":
    build()
    sys.exit(0)
