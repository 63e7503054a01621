"""Builds libattnsink.so in-tree with nvcc for sm_100a, and the Python binding
of its shortest calls (_binding.so, g++, against torch's headers).  Where only the
binding cannot be built, build() warns and the library is there all the same;
the calls that go through the binding then say what is missing.

Usage:  python -m sliding_window_learned_b200.build [--verbose-ptxas]
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libattnsink.so")
BINDING = os.path.join(HERE, "_binding.so")
BINDING_STAMP = os.path.join(BUILD, "binding.txt")   # binding_for() of the one that is there
SOURCES = ["api.cu", "api_cache.cu", "fwd_tc.cu", "fwd_cudacore.cu", "decode.cu", "decode_noalloc.cu",
           "decode_paged_fp8.cu", "cache_fp8.cu", "bwd.cu", "bwd_tc.cu"]
HEADERS = ["ptx.cuh", "status.cuh", "e4m3.cuh", "kernels.h", "api_internal.h"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    deps.append(os.path.join(os.path.dirname(HERE), "include", "attnsink.h"))
    return any(os.path.getmtime(p) > t for p in deps if os.path.exists(p))


def binding_for() -> str:
    """What a binding is built against: its headers and ABI are these versions' own."""
    import torch
    return (f"torch {torch.__version__} python {sys.version_info[0]}.{sys.version_info[1]} "
            f"cxx11abi {int(torch._C._GLIBCXX_USE_CXX11_ABI)}")


def _binding_stale() -> bool:
    src = os.path.join(CSRC, "binding.cpp")
    header = os.path.join(os.path.dirname(HERE), "include", "attnsink.h")
    if not os.path.exists(BINDING) or os.path.getmtime(BINDING) <= max(os.path.getmtime(src), os.path.getmtime(header)):
        return True
    try:
        with open(BINDING_STAMP) as f:
            return f.read() != binding_for()
    except OSError:
        return True


def build_binding(force: bool = False) -> str:
    """_binding.so: csrc/binding.cpp against torch's headers and libattnsink.so.
    Built again when a source, torch or Python is another one."""
    if not force and not _binding_stale():
        return BINDING
    import torch
    top = os.path.dirname(torch.__file__)
    nvcc = _nvcc()
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DATTN_SINK_BUILT_FOR="{binding_for()}"',
           "-isystem", os.path.join(top, "include"),
           "-isystem", os.path.join(top, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include"),
           "-isystem", sysconfig.get_paths()["include"], os.path.join(CSRC, "binding.cpp"), "-o", tmp,
           "-L", HERE, "-l:libattnsink.so", "-Wl,-rpath,$ORIGIN",
           "-L", os.path.join(top, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        failed = r.stderr if r.returncode != 0 else None
    except OSError as e:
        failed = str(e)
    if failed is not None:
        if os.path.exists(BINDING):        # (the old one's calls may not be the library's any more)
            os.remove(BINDING)
        raise RuntimeError(f"binding build failed:\n{failed}")
    os.replace(tmp, BINDING)
    os.makedirs(os.path.dirname(BINDING_STAMP), exist_ok=True)
    with open(BINDING_STAMP, "w") as f:
        f.write(binding_for())
    return BINDING


def _build_library(ptxas_verbose: bool) -> None:
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    common = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "--expt-relaxed-constexpr", "-I", CSRC]
    if ptxas_verbose:
        common += ["-Xptxas", "-v"]

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [nvcc, *common, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
        if ptxas_verbose:
            sys.stderr.write(r.stderr)
        return obj

    with concurrent.futures.ThreadPoolExecutor(len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart_static", "-ldl",
                        "-lrt", "-lpthread"], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)


def build(force: bool = False, ptxas_verbose: bool = False) -> str:
    """libattnsink.so, and _binding.so where its tools are there."""
    if force or _stale():
        _build_library(ptxas_verbose)
    try:
        build_binding(force)
    except Exception as e:
        warnings.warn(f"_binding.so is not built, the calls that go through it are not available: {e}",
                      RuntimeWarning, stacklevel=2)
    return LIB


if __name__ == "__main__":
    print(build(force=True, ptxas_verbose="--verbose-ptxas" in sys.argv))
