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
import warnings

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


def _sources(out: str):
    kinds = ("*.cpp",) if out == BINDING else ("*.cu", "*.cuh")
    return sorted([s for k in kinds for s in glob.glob(os.path.join(CSRC, k))] + glob.glob(os.path.join(INCLUDE, "*.h")))


def _newer_than_sources(out: str) -> bool:
    return os.path.exists(out) and all(os.path.getmtime(s) <= os.path.getmtime(out) for s in _sources(out))


def up_to_date() -> bool:
    return _newer_than_sources(LIB) and _newer_than_sources(BINDING)


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
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            f'-DBL_TORCH_VERSION="{torch.__version__}"', "-I", INCLUDE,
            *(f for i in include for f in ("-isystem", i)), os.path.join(CSRC, "attn_binding.cpp"), "-o", out,
            "-L" + libs, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath," + libs]


def _run(cmd):
    """A compiler started -> a function that waits for it and gives (ok, output)."""
    try:
        job = subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    except OSError as e:
        failed = f"{cmd[0]}: {e}\n"
        return lambda: (False, failed)

    def wait():
        out, _ = job.communicate()
        return job.returncode == 0, out

    return wait


def build(force: bool = False, verbose: bool = False) -> str:
    nvcc = os.environ.get("NVCC", "nvcc")
    lib = host = None
    if force or not _newer_than_sources(LIB):
        lib = _run([nvcc, *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, *sorted(glob.glob(os.path.join(CSRC, "*.cu"))),
                    "-o", LIB + ".tmp", "-lcuda"])
    if force or not _newer_than_sources(BINDING):
        host = _run(_binding_cmd(nvcc, BINDING + ".tmp"))
    host_ok, host_out = host() if host else (True, "")
    if lib:
        ok, out = lib()
        if not ok:
            sys.stderr.write(out)
            raise RuntimeError("nvcc failed building libbitlinear.so")
        if verbose:
            sys.stderr.write(out)
        os.replace(LIB + ".tmp", LIB)
    if host and host_ok:
        os.replace(BINDING + ".tmp", BINDING)
    elif host:
        # the library does without it; one of older sources must not stay behind
        if os.path.exists(BINDING):
            os.remove(BINDING)
        warnings.warn("attn_binding.so was not built (attention calls take 5 to 10 us longer on the host):\n" + host_out,
                      RuntimeWarning, stacklevel=2)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
