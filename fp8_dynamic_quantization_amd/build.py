"""Build libhq.so (the C-ABI library) for gfx950 with hipcc, in-tree, and the
native torch binding _hqtorch.so (host code only) beside it.

    python -m fp8_dynamic_quantization_amd.build

Every HIP source is compiled with packed-fp32 instruction selection disabled
(``-Xclang -target-feature -Xclang -packed-fp32-ops``); the fp32 division used
for scales stays correctly rounded (hipcc's default) and fp32 denormals are kept.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libhq.so")
BINDING = os.path.join(PKG, "_hqtorch.so")

SOURCES = ["quantize.hip", "gemm.hip", "gemm_fused.hip", "blockscaled.hip", "norm.hip", "act.hip", "wgrad.hip", "moe.hip", "probe.hip",
           "hq_api.cpp"]

# Per-source flags. The GEMM keeps its MFMA accumulators in VGPRs and the
# operand fragments in AGPRs: with 256 accumulator registers per wavefront the
# default AGPR-accumulator allocation spills to scratch, this form does not.
EXTRA = {src: ["-mllvm", "-amdgpu-mfma-vgpr-form=1"] for src in ("gemm.hip", "gemm_fused.hip", "blockscaled.hip", "wgrad.hip", "moe.hip")}

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
COMMON = [
    f"--offload-arch={ARCH}", "-O3", "-fPIC", "-std=c++17",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-result",
    "-I", INCLUDE, "-I", CSRC,
]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *COMMON, *EXTRA.get(src, []), "-x", "hip", "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj


def _compile_binding() -> str:
    """The binding's object: a CPython module against torch's C++ headers."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    obj = os.path.join(BUILD, "torch_binding.o")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-fPIC", "-std=c++17", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
           "-I", INCLUDE, *(f"-isystem{p}" for p in cpp_extension.include_paths()), "-isystem/opt/rocm/include",
           f"-isystem{sysconfig.get_paths()['include']}", "-c", os.path.join(CSRC, "torch_binding.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compiling torch_binding.cpp failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj


def _link(cmd: list[str], out: str) -> None:
    r = subprocess.run([*cmd, "-o", out + ".tmp"], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(out + ".tmp", out)


def _link_binding(obj: str) -> None:
    from torch.utils import cpp_extension

    # torch's libraries are in the process already when the binding is imported
    torch_lib = os.path.join(os.path.dirname(cpp_extension.__file__), "..", "lib")
    _link([os.environ.get("CXX", "g++"), "-shared", obj, f"-L{PKG}", "-l:libhq.so", f"-L{torch_lib}", "-lc10", "-lc10_hip",
           "-ltorch_cpu", "-ltorch_hip", "-ltorch_python", "-Wl,-rpath,$ORIGIN"], BINDING)


def build(verbose: bool = False) -> str:
    """Compile every source and link libhq.so and the binding; returns the library path.

    The C library needs neither torch nor a host compiler: it is linked before the
    binding's object is waited for, so a failure there leaves it built (and raises)."""
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_compile_binding)
        objs = list(ex.map(_compile, SOURCES))
        _link([HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-Wl,-soname,libhq.so", *objs], LIB)
        _link_binding(binding.result())
    if verbose:
        print(f"built {LIB}")
    return LIB


def clean() -> None:
    shutil.rmtree(BUILD, ignore_errors=True)


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
