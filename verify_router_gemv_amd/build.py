"""Compile the HIP library in-tree, verify_router_gemv_amd/libmoe_round.so (gfx950), and the extension module
_verify_ops.so that binds the verify-round operators to Python.

    python -m verify_router_gemv_amd.build [--verbose]
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import time

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libmoe_round.so")
MODULE = os.path.join(PKG, "_verify_ops.so")
SOURCES = (["moe_round.hip", "moe_validate.cpp", "verify_ops.hip", "verify_attention_bf16.hip",
            "verify_attention_f16.hip", "verify_validate.cpp"] + [f"moe_gemv_g{g}.hip" for g in (4, 8, 16, 32, 64)]
           + [f"moe_gemv_g{g}_s256.hip" for g in (4, 8, 16, 32, 64)])

ARCH = "gfx950"
FLAGS = [
    "-O3", "-std=c++17", "-fPIC",
    f"--offload-arch={ARCH}",
    "-munsafe-fp-atomics",                      # hardware fp32 atomic add for the scatter-add
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",   # no packed fp32 VALU ops
    "-fvisibility=hidden",
    "-Wall", "-Wno-unused-result",
]
# Per-source flags. moe_round.hip holds the prefill GEMMs, whose matrix-core results are folded
# into the accumulators on the vector ALUs: with the results in ordinary VGPRs (not accumulation
# registers) that costs no register-to-register copies. Its other matrix-core kernel (the fp64
# router GEMM) only stores its results.
SOURCE_FLAGS = {"moe_round.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"],
                "moe_gemv_g16.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"],  # the down tile's results fold on VALU
                # the scores are masked and exponentiated, the outputs rescaled, on the vector ALUs
                "verify_attention_bf16.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"],
                "verify_attention_f16.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"]}


def hipcc() -> str:
    for cand in (shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found; the HIP library cannot be built")


def _compile(src: str, obj: str) -> None:
    cmd = [hipcc(), *FLAGS, *SOURCE_FLAGS.get(src, []), f"-I{INCLUDE}", "-c", os.path.join(CSRC, src), "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"hipcc failed ({res.returncode}): {' '.join(cmd)}")


def _compile_module(obj: str) -> None:
    """The binding: host code over torch's C++ headers."""
    import sysconfig

    from torch.utils.cpp_extension import include_paths
    inc = [f"-I{INCLUDE}", f"-I{sysconfig.get_paths()['include']}"]
    for d in include_paths("cuda"):
        inc += ["-isystem", d]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-Wall", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
           *inc, "-c", os.path.join(CSRC, "verify_binding.cpp"), "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"g++ failed ({res.returncode}): {' '.join(cmd)}")


def _link_module(obj: str) -> None:
    import torch
    tlib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = MODULE + ".tmp"
    cmd = ["g++", "-shared", "-o", tmp, obj, f"-L{tlib}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_hip",
           f"-L{PKG}", "-l:libmoe_round.so", "-Wl,-rpath,$ORIGIN"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"link failed ({res.returncode}): {' '.join(cmd)}")
    os.replace(tmp, MODULE)


def build(verbose: bool = False, jobs: int = 0) -> str:
    """Compile every translation unit in parallel, then link the shared library."""
    from concurrent.futures import ThreadPoolExecutor
    t0 = time.time()
    objdir = os.path.join(PKG, "_build")
    os.makedirs(objdir, exist_ok=True)
    objs = [os.path.join(objdir, os.path.splitext(s)[0] + ".o") for s in SOURCES]
    jobs = jobs or min(len(SOURCES), max(1, (os.cpu_count() or 4)))
    binding = os.path.join(objdir, "verify_binding.o")
    with ThreadPoolExecutor(max_workers=jobs) as pool:
        for f in [pool.submit(_compile, s, o) for s, o in zip(SOURCES, objs)] + [pool.submit(_compile_module, binding)]:
            f.result()
    tmp = LIB + ".tmp"
    cmd = [hipcc(), "-shared", "-fPIC", f"--offload-arch={ARCH}", "-o", tmp] + objs
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"link failed ({res.returncode}): {' '.join(cmd)}")
    os.replace(tmp, LIB)
    _link_module(binding)
    if verbose:
        print(f"built {LIB} in {time.time() - t0:.1f}s")
    return LIB


if __name__ == "__main__":
    build(verbose="--verbose" in sys.argv or "-v" in sys.argv)
