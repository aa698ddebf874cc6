"""Build the CUDA library (libssm_gb300.so) in-tree with nvcc for sm_103a.

Each .cu under csrc/ compiles to an object in parallel, then one shared library is linked
with the CUDA runtime statically.  Rebuilds only when a source or header is newer than the
library.  build(debug=True) makes the debug library (libssm_gb300_debug.so, -DSSM_DEBUG): the
same kernels with their device index checks compiled in (see ssm_debug_build in ssm.h).
build_binding() makes the compiled part of the Python entry points in _layer.py.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libssm_gb300.so")
BUILD_DEBUG = os.path.join(HERE, "_build_debug")
LIB_DEBUG = os.path.join(HERE, "libssm_gb300_debug.so")

BINDING = os.path.join(HERE, "_binding.so")
BINDING_KEY = os.path.join(BUILD, "binding.key")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-I", INCLUDE] + ARCH


def nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found: the CUDA library cannot be built")
    return exe


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale(lib) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    return any(os.path.getmtime(f) > t for f in deps)


def build(force: bool = False, verbose: bool = False, debug: bool = False) -> str:
    lib, bdir = (LIB_DEBUG, BUILD_DEBUG) if debug else (LIB, BUILD)
    if not force and not _stale(lib):
        return lib
    os.makedirs(bdir, exist_ok=True)
    exe = nvcc()
    flags = NVCC_FLAGS + (["-DSSM_DEBUG"] if debug else [])

    def compile_one(src):
        obj = os.path.join(bdir, os.path.basename(src)[:-3] + ".o")
        cmd = [exe, *flags, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        results = list(ex.map(compile_one, sources()))
    if verbose:
        for _, log in results:
            print(log)
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [exe, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results], "-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


def build_binding(force: bool = False) -> str:
    """Build the compiled Python entry points of the operators around a layer's scan (_binding.so, from
    csrc/binding.cpp) with g++ against the installed torch.

    It holds inline code and object layouts of the torch and Python that it was compiled with, so a key beside it (their
    versions and the command) says which they were; with others, or without a key, it is built anew."""
    import sysconfig

    import torch
    src = os.path.join(CSRC, "binding.cpp")
    home = os.path.dirname(torch.__file__)
    inc = [sysconfig.get_path("include"), os.path.join(home, "include"),
           os.path.join(home, "include", "torch", "csrc", "api", "include")]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", *[f"-I{p}" for p in inc],
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", src,
           f"-L{os.path.join(home, 'lib')}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]
    key = "\n".join([torch.__version__, str(torch.version.git_version), str(sysconfig.get_config_var("EXT_SUFFIX")), *cmd])
    if not force and _binding_is_current(src, key):
        return BINDING
    os.makedirs(BUILD, exist_ok=True)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")  # (needed to build only)
    tmp = BINDING + f".tmp{os.getpid()}"
    r = subprocess.run([*cmd, f"-I{cuda}", "-o", tmp], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on binding.cpp:\n{r.stdout}\n{r.stderr}")
    if os.path.exists(BINDING_KEY):
        os.remove(BINDING_KEY)  # never a new key beside an old module
    os.replace(tmp, BINDING)
    with open(BINDING_KEY + f".tmp{os.getpid()}", "w") as f:
        f.write(key)
    os.replace(f.name, BINDING_KEY)
    return BINDING


def _binding_is_current(src, key) -> bool:
    if not os.path.exists(BINDING) or not os.path.exists(BINDING_KEY):
        return False
    with open(BINDING_KEY) as f:
        if f.read() != key:
            return False
    built = os.path.getmtime(BINDING)
    return all(os.path.getmtime(p) <= built for p in [src, *glob.glob(os.path.join(INCLUDE, "*.h"))])


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, debug="--debug" in sys.argv))
