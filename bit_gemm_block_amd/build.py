"""Builds libw4a4.so (HIP kernels + C ABI) for gfx950 with hipcc, in-tree, and,
where torch is installed, _block.so, the Python binding of its operators beside
the layer and of a decoding step (host code against torch's headers).

    python -m bit_gemm_block_amd.build
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libw4a4.so")
BINDING = os.path.join(PKG, "_block.so")

SOURCES = ["api.cpp", "rotq.hip", "rotq_mfma.hip", "qgemm.hip", "qgemm_f6.hip", "lowrank.hip", "offq.hip",
           "noalloc.hip", "block_api.cpp", "adapters.hip", "norm_residual.hip", "gated.hip",
           "decode_api.cpp", "w4a16.hip", "cache.hip", "attention.hip", "attention_d64.hip", "attention_d128.hip",
           "attention_d256.hip"]

# No fast-math and no denormal flushing: the quantizer's float32 division and
# rounding must follow IEEE.  Packed-FP32 instructions are disabled.
HIP_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
]


def hipcc() -> str:
    for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("hipcc not found")


def _compile(src: str, extra: list[str]) -> str:
    obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
    lang = ["-x", "hip"] if src.endswith(".hip") else []
    cmd = [hipcc()] + HIP_FLAGS + extra + ["-I", INCLUDE, "-I", CSRC] + lang + \
          ["-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj


def _binding() -> str | None:
    """Object file of the binding (None without torch)."""
    import sysconfig

    try:
        from torch.utils import cpp_extension
    except ImportError as e:
        print(f"{os.path.basename(BINDING)}, the Python binding of the operators beside the layer, needs torch "
              f"and is not built ({e})")
        return None
    obj = os.path.join(BUILD_DIR, "block_binding.cpp.o")
    rocm = os.path.join(os.path.dirname(os.path.dirname(hipcc())), "include")
    cxx = os.environ.get("CXX") or shutil.which("g++") or hipcc()
    cmd = [cxx, "-x", "c++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1", "-I", INCLUDE]
    for i in cpp_extension.include_paths() + [sysconfig.get_paths()["include"], rocm]:
        cmd += ["-isystem", i]
    cmd += ["-c", os.path.join(CSRC, "block_binding.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compiler failed for block_binding.cpp:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj


def _link(out: str, args: list[str]) -> None:
    tmp = out + ".tmp"
    cmd = [hipcc(), "-shared", "-fPIC", "-o", tmp] + args
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)


def link_binding(obj: str) -> None:
    """_block.so beside libw4a4.so, which it calls."""
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    _link(BINDING, [obj, "-L", PKG, "-l:libw4a4.so", "-Wl,-rpath,$ORIGIN", "-L", lib, "-ltorch_python",
                    "-ltorch_cpu", "-lc10", "-lc10_hip"])


def build(extra: list[str] | None = None, save_temps: bool = False) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    extra = list(extra or [])
    if save_temps:
        extra += ["-save-temps=obj"]
    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_binding)
        objs = list(ex.map(lambda s: _compile(s, extra), SOURCES))
        _link(LIB, ["--offload-arch=gfx950"] + objs)
        obj = binding.result()
        if obj:
            link_binding(obj)
    return LIB


if __name__ == "__main__":
    print(build(save_temps="--save-temps" in sys.argv))
