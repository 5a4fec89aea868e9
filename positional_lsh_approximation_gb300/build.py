"""Build libplsh.so (the C-ABI library) in-tree with nvcc for sm_103a.

Each translation unit is compiled in parallel, then linked into one shared
library next to this file (`_build/libplsh.so`).  The native binding of the
4-bit cache's calls (`_build/_plsh_binding.so`, a Python extension against
torch's headers) is compiled beside them and linked to it; where it cannot be
(no torch, no Python headers, no host compiler), the library is built all the
same, a warning says why, and the 4-bit cache's calls raise.  No CMake.
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
SRC_DIR = os.path.join(HERE, "csrc")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(BUILD_DIR, "libplsh.so")
SOURCES = ["api.cu", "sampler.cu", "attn_simt.cu", "attn_tc.cu", "decode.cu", "bias.cu", "bwd.cu",
           "bwd_tc.cu", "q4_cache.cu", "q4_decode.cu", "q4_pages.cu",
           "q4_many.cu"]
BINDING_PATH = os.path.join(BUILD_DIR, "_plsh_binding.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
         "-Xcompiler", "-ffp-contract=off", "--expt-relaxed-constexpr"]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required")
    return path


def _stale(obj: str, src: str) -> bool:
    if not os.path.exists(obj):
        return True
    deps = [src] + [os.path.join(SRC_DIR, f) for f in os.listdir(SRC_DIR)
                    if f.endswith((".h", ".cuh"))]
    deps.append(os.path.join(HERE, "..", "include", "plsh.h"))
    return any(os.path.getmtime(d) > os.path.getmtime(obj) for d in deps)


def _torch_dir() -> str:
    import torch
    return os.path.dirname(torch.__file__)


def _binding_compile(out: str) -> list:
    import torch
    t = os.path.join(_torch_dir(), "include")
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    return [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-I" + t, "-I" + os.path.join(t, "torch", "csrc", "api", "include"),
            "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(cuda, "include"),
            "-c", os.path.join(SRC_DIR, "binding.cpp"), "-o", out]


def _binding_link(obj: str, out: str) -> list:
    return [shutil.which("g++") or "g++", "-shared", "-o", out, obj,
            "-L" + os.path.join(_torch_dir(), "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu",
            "-ltorch_cuda", "-lc10", "-lc10_cuda", "-L" + BUILD_DIR, "-lplsh",
            "-Wl,-rpath,$ORIGIN"]


def binding_abi() -> str:
    """What a binding compiled now would be for."""
    import torch
    return f"torch {torch.__version__}, C++11 ABI {int(torch._C._GLIBCXX_USE_CXX11_ABI)}, " \
           f"Python {sysconfig.get_config_var('SOABI')}"


def built_binding_abi():
    """What the binding was compiled for, or None: it is of no use to another
    torch, whose tensors are laid out otherwise."""
    try:
        with open(BINDING_PATH + ".for") as f:
            return f.read()
    except FileNotFoundError:
        return None


def _run_host(cmd: list) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("compiler failed: " + " ".join(cmd) + "\n" + r.stdout + r.stderr)


def _compile_binding(force: bool):
    """The binding's object if it is to be linked anew, else None."""
    obj = os.path.join(BUILD_DIR, "binding.o")
    if force or _stale(obj, os.path.join(SRC_DIR, "binding.cpp")) or built_binding_abi() != binding_abi():
        if os.path.exists(obj):
            os.remove(obj)
        _run_host(_binding_compile(obj))
    elif os.path.exists(BINDING_PATH):
        return None
    return obj


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    nv = nvcc()
    jobs = []
    for src in SOURCES:
        s = os.path.join(SRC_DIR, src)
        o = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        if force or _stale(o, s):
            cmd = [nv, *ARCH, *FLAGS, *extra, "-c", s, "-o", o]
            if verbose:
                cmd.insert(1, "-Xptxas=-v")
            jobs.append(cmd)

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_compile_binding, force)
        for cmd, r in ex.map(run, jobs):
            if verbose or r.returncode != 0:
                print(r.stdout + r.stderr)
            if r.returncode != 0:
                raise RuntimeError("nvcc failed: " + " ".join(cmd))
    objs = [os.path.join(BUILD_DIR, s.replace(".cu", ".o")) for s in SOURCES]
    if jobs or not os.path.exists(LIB_PATH):
        tmp = LIB_PATH + f".tmp{os.getpid()}"
        cmd = [nv, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
        os.replace(tmp, LIB_PATH)
    try:
        obj = binding.result()
        if obj is not None:
            tmp = BINDING_PATH + f".tmp{os.getpid()}"
            _run_host(_binding_link(obj, tmp))
            if os.path.exists(BINDING_PATH + ".for"):
                os.remove(BINDING_PATH + ".for")
            os.replace(tmp, BINDING_PATH)
            with open(BINDING_PATH + ".for", "w") as f:
                f.write(binding_abi())
    except (ImportError, OSError, RuntimeError) as e:
        if os.path.exists(BINDING_PATH):          # of other sources
            os.remove(BINDING_PATH)
        warnings.warn(f"the native binding of the 4-bit cache's calls was not built: {e}",
                      RuntimeWarning, stacklevel=2)
    return LIB_PATH


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
