"""Build libsdpa.so in-tree with nvcc for sm_103a (GB300).

Each CUDA translation unit under ``csrc/`` is compiled in parallel into
``_build/`` and linked into ``libsdpa.so`` next to this file. The CUDA runtime
is linked statically; the driver entry point for TMA descriptor encoding is
looked up at run time, so the library loads on machines without a GPU.
``_binding.so``, the native binding of the calls with the shortest kernels, is
compiled by g++ against torch's headers and linked to that library. Where torch is
not installed it is left out: the library and its C entry points do not need it.
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libsdpa.so")
BINDING = os.path.join(HERE, "_binding.so")
SOURCES = ["api.cu", "aux.cu", "noalloc.cu", "fwd_bf16.cu", "fwd_fp16.cu", "bwd_dkdv_bf16.cu",
           "bwd_dkdv_fp16.cu", "bwd_dq_bf16.cu", "bwd_dq_fp16.cu", "bwd_fused_bf16.cu",
           "bwd_fused_fp16.cu", "fwd_cap.cu", "bwd_dkdv_cap_bf16.cu", "bwd_dkdv_cap_fp16.cu",
           "bwd_dq_cap.cu", "bwd_fused_cap.cu", "norm_rope.cu", "norm_rope_api.cu",
           "prefix_bf16.cu", "prefix_fp16.cu", "prefix_join.cu", "page_slots.cu",
           "paged_bf16.cu", "paged_fp16.cu", "paged_join.cu", "paged_api.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr"]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found; the CUDA 13 toolkit is required to build libsdpa.so")
    return cand


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *ARCH, *FLAGS, "-I", os.path.join(HERE, "..", "include"), "-c",
           os.path.join(CSRC, src), "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if verbose and r.stderr:
        sys.stderr.write(r.stderr)
    return obj


def _run(cmd: list[str], what: str) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _torch():
    """The installed torch, or None."""
    try:
        import torch
    except ImportError:
        return None
    return torch


def _compile_binding(torch) -> str:
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    obj = os.path.join(BUILD, "binding.o")
    _run(["g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          f'-DSDPA_TORCH_VERSION="{torch.__version__}"',
          "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
          "-isystem", sysconfig.get_paths()["include"], "-isystem", cuda, "-c", os.path.join(CSRC, "binding.cpp"),
          "-o", obj], "g++ on binding.cpp")
    return obj


def _link_binding(torch, obj: str) -> None:
    torch_lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    _run(["g++", "-shared", "-o", BINDING + ".tmp", obj, "-L" + HERE, "-l:libsdpa.so",
          "-L" + torch_lib, "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda",
          "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + torch_lib], "link of _binding.so")
    os.replace(BINDING + ".tmp", BINDING)


def build(verbose: bool = False, jobs: int | None = None) -> str:
    """Compile every translation unit and link libsdpa.so; returns its path."""
    os.makedirs(BUILD, exist_ok=True)
    jobs = jobs or min(len(SOURCES) + 1, os.cpu_count() or 1)
    torch = _torch()
    with concurrent.futures.ThreadPoolExecutor(max_workers=jobs) as ex:
        binding = None if torch is None else ex.submit(_compile_binding, torch)
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "--cudart", "static", "-o", tmp, *objs]
    _run(cmd, "link of libsdpa.so")
    os.replace(tmp, LIB)
    # the library is there whatever becomes of the binding, and no binding of another build beside it
    if os.path.exists(BINDING):
        os.remove(BINDING)
    if binding is None:
        sys.stderr.write("torch is not installed: libsdpa.so is built, _binding.so is left out\n")
    else:
        _link_binding(torch, binding.result())
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
