"""Build libgdn.so (all HIP kernels + the C ABI) for gfx950 with hipcc, and
_binding.so (the Python binding of the block operators) with the host compiler.

Usage: python -m linear_attention_token_conv1d_amd._build
Objects go to _build/ at the repository root; the libraries are written next
to this file so they travel with the source tree.
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
OUT = os.path.join(PKG, "libgdn.so")
BINDING = os.path.join(PKG, "_binding.so")
BUILD = os.path.join(ROOT, "_build")
ARCH = "gfx950"

SOURCES = ["gdn_api.cpp", "conv1d.hip", "decode.hip", "prefill.hip", "backward.hip", "probe.hip",
           "block_api.cpp", "norm.hip", "rope.hip", "kv_cache.hip", "attention.hip"]

FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-fPIC",
    "-std=c++17",
    "-Wall",
    "-Wno-unused-function",
    # packed-fp32 instructions are kept off (plain fp32 VALU code only)
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # MFMA accumulators live in ordinary VGPRs: the scan's accumulator tiles
    # feed VALU math every chunk, and AGPR copies would double that traffic
    "-mllvm", "-amdgpu-mfma-vgpr-form",
    "-I", os.path.join(ROOT, "include"),
]


def hipcc():
    exe = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(exe):
        raise RuntimeError("hipcc not found; a ROCm toolchain is required to build libgdn.so")
    return exe


def _compile(src, verbose):
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [hipcc(), *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    if src.endswith(".cpp"):
        cmd[1:1] = ["-x", "hip"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if r.stderr.strip() and verbose:
        print(r.stderr, file=sys.stderr)
    return obj


def _run(cmd, what, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _binding(verbose):
    """_binding.so: host code only; it links libgdn.so, which lies beside it, and torch's libraries, which the
    process that imports it has loaded."""
    import sysconfig

    import torch

    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        raise RuntimeError("no host C++ compiler found for _binding.so")
    t = os.path.dirname(torch.__file__)
    tmp = BINDING + ".tmp"
    _run([cxx, "-shared", "-fPIC", "-std=c++17", "-O2", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM", "-isystem", os.path.join(t, "include"), "-isystem",
          os.path.join(t, "include", "torch", "csrc", "api", "include"), "-isystem", sysconfig.get_paths()["include"],
          os.path.join(CSRC, "binding.cpp"), "-o", tmp, "-L", os.path.join(t, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10",
          "-L", PKG, "-l:libgdn.so", "-Wl,-rpath,$ORIGIN"], "binding.cpp", verbose)
    os.replace(tmp, BINDING)


def build(verbose=False):
    """Compile every source and link libgdn.so and _binding.so.  Always rebuilds."""
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(4, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    tmp = OUT + ".tmp"
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    _run(cmd, "link", verbose)
    os.replace(tmp, OUT)
    _binding(verbose)
    return OUT


if __name__ == "__main__":
    print(build(verbose=True))
