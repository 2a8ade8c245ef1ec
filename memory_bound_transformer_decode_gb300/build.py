"""Builds the decode library (csrc/*.cu) for sm_103a into _build/libddl.so, and
the module of its per-layer calls for torch tensors (csrc/ddl_torch.cpp) into
_build/_ddl_torch.so, which links against it.  Without torch the library alone
is built (``python build.py``), with nothing but nvcc.

Plain nvcc and g++, one translation unit per file compiled in parallel, then the
shared-library links; no CMake.  ``ddl.py`` loads the library with ctypes and
imports the module.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libddl.so")
TORCH_SRC = os.path.join(CSRC, "ddl_torch.cpp")
TORCH_LIB = os.path.join(BUILD, "_ddl_torch.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-Xptxas", "-v"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build the library")
    return cand


def _torch_dirs() -> tuple[list[str], str] | None:
    """Include directories and the library directory of the installed torch;
    None where there is none: the C library is built all the same."""
    try:
        import torch
    except ImportError:
        return None
    root = os.path.dirname(torch.__file__)
    inc = os.path.join(root, "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    return [inc, os.path.join(inc, "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"],
            cuda], os.path.join(root, "lib")


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _stale(out: str, deps: list[str]) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    api = os.path.join(HERE, "..", "include", "ddl.h")
    srcs = sources()
    lib = force or _stale(LIB, srcs + headers + [api, __file__])
    module = force or _stale(TORCH_LIB, [TORCH_SRC, api, __file__])
    dirs = _torch_dirs() if module else None
    if not lib and not dirs:
        return LIB
    nvcc = _nvcc() if lib else ""
    tobj = os.path.join(BUILD, "ddl_torch.o")

    def compile_one(src: str) -> tuple[str, str]:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    def compile_torch() -> None:
        cmd = ["g++", "-O2", "-std=c++20", "-fPIC", *[f"-I{i}" for i in dirs[0]], "-c", TORCH_SRC, "-o", tobj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed on {TORCH_SRC}:\n{r.stdout}\n{r.stderr}")

    with cf.ThreadPoolExecutor(max_workers=len(srcs) + 1) as ex:
        binding = ex.submit(compile_torch) if dirs else None
        results = list(ex.map(compile_one, srcs)) if lib else []
        if lib:
            _link(LIB, [nvcc, *ARCH, "-shared"], [o for o, _ in results])
        if binding:  # (the library does not need it: its own link comes first)
            binding.result()
            _link(TORCH_LIB, ["g++", "-shared"],
                  [tobj, f"-L{BUILD}", "-lddl", f"-L{dirs[1]}", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
                   "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{dirs[1]}"])
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    if lib:
        with open(os.path.join(BUILD, "ptxas.log"), "w") as f:
            for _, log in results:
                f.write(log)
    return LIB


def _link(out: str, linker: list[str], inputs: list[str]) -> None:
    tmp = out + f".tmp{os.getpid()}"
    r = subprocess.run([*linker, "-o", tmp, *inputs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
