"""Builds libconvrot.so (all gfx950 HIP kernels and the C-ABI host layer) with
hipcc, and _native (the CPython side of some entry points, for this Python and
this torch) with g++, both in-tree. Every call recompiles."""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libconvrot.so")
# named for the interpreter, so that no other one loads it: it uses more than the stable interface
NATIVE = os.path.join(HERE, "_native" + sysconfig.get_config_var("EXT_SUFFIX"))
SOURCES = ["rq.hip", "pack.hip", "merge.hip", "gemm_w4a4.hip", "gemm_int.hip", "gemm_w4a8.hip", "gemm_f6.hip", "abi.cpp",
           "lora.hip", "act.hip", "adapter_abi.cpp", "mx.hip", "gemm_mx.hip", "norm.hip", "adamw.hip", "block_abi.cpp"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "-O3", "-std=c++17", "-fPIC", "--offload-arch=gfx950",
    "-ffp-contract=off",
    # matrix-core accumulators stay in arch VGPRs (no per-MFMA AGPR copies of
    # loop-carried accumulators)
    "-mllvm", "-amdgpu-mfma-vgpr-form",
    # packed fp32 VALU ops stay off: hipcc would otherwise form them from float code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
]


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *FLAGS, "-x", "hip", "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if verbose and r.stderr.strip():
        noise = "is not a recognized feature for this target"
        lines = [ln for ln in r.stderr.splitlines() if noise not in ln]
        if lines:
            print("\n".join(lines))
    return obj


def _compile_binding() -> str:
    """binding.cpp against the torch that is installed."""
    import torch
    from torch.utils.cpp_extension import include_paths
    obj = os.path.join(BUILD, "binding.o")
    rocm = os.path.dirname(os.path.dirname(HIPCC))
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-Wno-attributes", "-D__HIP_PLATFORM_AMD__",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", f'-DBUILT_FOR_TORCH="{torch.__version__}"',
           *[f"-isystem{p}" for p in (*include_paths(), sysconfig.get_paths()["include"], os.path.join(rocm, "include"))],
           "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for binding.cpp:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_binding(obj: str) -> None:
    import torch
    from torch.utils.cpp_extension import library_paths
    dirs = library_paths()
    tmp = NATIVE + ".tmp"
    cmd = ["g++", "-shared", "-fPIC", obj, "-o", tmp, f"-L{HERE}", "-l:libconvrot.so", "-Wl,-rpath,$ORIGIN",
           *[f"-L{d}" for d in dirs], "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_hip"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, NATIVE)
    unnamed = os.path.join(HERE, "_native.so")           # its earlier name, which any interpreter loads
    if os.path.exists(unnamed):
        os.remove(unnamed)


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(len(SOURCES) + 1, os.cpu_count() or 4)) as ex:
        binding = ex.submit(_compile_binding)
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, "-shared", "-fPIC", "--offload-arch=gfx950", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _link_binding(binding.result())
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
