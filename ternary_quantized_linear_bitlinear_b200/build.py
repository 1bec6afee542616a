"""Build libbitlinear.so (sm_100a, nvcc) and attn_binding.so (host code over
torch's headers, g++) in-tree.

    python -m ternary_quantized_linear_bitlinear_b200.build [--force]
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libbitlinear.so")
BINDING = os.path.join(PKG, "attn_binding.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-shared", "-Xcompiler", "-fPIC,-O2",
    "--expt-relaxed-constexpr",
    "--threads", "2",
    "-Xptxas", "-v",
]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp"))
                  + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(INCLUDE, "*.h")))


def up_to_date() -> bool:
    if not (os.path.exists(LIB) and os.path.exists(BINDING)):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    return all(os.path.getmtime(s) <= t for s in _sources())


def _binding_cmd(nvcc: str, out: str):
    import torch

    base = os.path.dirname(os.path.abspath(torch.__file__))
    found = shutil.which(nvcc)
    cuda = os.environ.get("CUDA_HOME") or (os.path.dirname(os.path.dirname(os.path.realpath(found))) if found
                                           else "/usr/local/cuda")
    include = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
               os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    libs = os.path.join(base, "lib")
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
            *(f for i in include for f in ("-isystem", i)), os.path.join(CSRC, "attn_binding.cpp"), "-o", out,
            "-L" + libs, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath," + libs]


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    nvcc = os.environ.get("NVCC", "nvcc")
    cmd = [nvcc, *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, *sorted(glob.glob(os.path.join(CSRC, "*.cu"))),
           "-o", LIB + ".tmp", "-lcuda"]
    host = subprocess.Popen(_binding_cmd(nvcc, BINDING + ".tmp"), stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                            text=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    host_out, _ = host.communicate()
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("nvcc failed building libbitlinear.so")
    if host.returncode != 0:
        sys.stderr.write(host_out)
        raise RuntimeError("g++ failed building attn_binding.so")
    if verbose:
        sys.stderr.write(res.stderr)
    os.replace(LIB + ".tmp", LIB)
    os.replace(BINDING + ".tmp", BINDING)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
