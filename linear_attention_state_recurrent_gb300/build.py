"""Builds libkda.so in-tree from csrc/*.cu for sm_103a (nvcc, one translation unit per
process, compiled in parallel, then linked into one shared library), and beside it
_kda_torch-<torch>-<python>.so from binding/kda_torch.cpp (the host compiler against the installed torch)."""
from __future__ import annotations

import concurrent.futures
import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libkda.so")
BINDING = os.path.join(PKG, "binding", "kda_torch.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I" + os.path.join(ROOT, "include")]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libkda")
    return path


def binding_lib() -> str:
    """The torch binding's file, named after the torch and the Python it is built against: one of another
    torch is not taken for it."""
    return os.path.join(PKG, f"_kda_torch-{importlib.metadata.version('torch')}-{sysconfig.get_config_var('SOABI')}.so")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + \
        sorted(glob.glob(os.path.join(CSRC, "*.h"))) + [os.path.join(ROOT, "include", "kda.h"),
                                                        BINDING, os.path.abspath(__file__)]


def up_to_date() -> bool:
    binding = binding_lib()
    if not os.path.exists(LIB) or not os.path.exists(binding):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(binding))
    return all(os.path.getmtime(d) <= t for d in _deps())


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _torch_dir():
    return os.path.dirname(importlib.util.find_spec("torch").origin)   # found, not imported


def _compile_binding():
    obj = os.path.join(OBJ, "kda_torch.o")
    torch_include = os.path.join(_torch_dir(), "include")
    cuda_include = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-c", BINDING, "-o", obj, "-I" + os.path.join(ROOT, "include"), "-I" + torch_include,
          "-I" + os.path.join(torch_include, "torch", "csrc", "api", "include"), "-I" + sysconfig.get_paths()["include"],
          "-I" + cuda_include], "compiling the torch binding")
    return obj


def _link_binding(obj):
    lib = os.path.join(_torch_dir(), "lib")
    tmp = binding_lib() + ".tmp"
    _run(["g++", "-shared", obj, "-o", tmp, "-L" + PKG, "-l:libkda.so", "-Wl,-rpath,$ORIGIN", "-L" + lib, "-ltorch_python", "-ltorch_cpu",
          "-lc10", "-lc10_cuda"], "linking the torch binding")
    os.replace(tmp, binding_lib())


def build(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    """Compile and link libkda.so and the torch binding; returns libkda.so's path. Raises on any compiler error."""
    if not force and up_to_date():
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    cc = nvcc()
    flags = ARCH + NVCC_FLAGS + list(extra_flags or [])

    def compile_one(src):
        obj = os.path.join(OBJ, os.path.basename(src) + ".o")
        cmd = [cc] + flags + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr)
        return obj

    srcs = _sources()
    with concurrent.futures.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 4))) as ex:
        binding = ex.submit(_compile_binding)
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + ".tmp"
    cmd = [cc] + ARCH + ["-shared", "-o", tmp] + objs + ["-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _link_binding(binding.result())   # libkda.so is there without it
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
