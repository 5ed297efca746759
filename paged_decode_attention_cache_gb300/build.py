"""Builds libpkv.so (the CUDA library behind include/pkv.h) in-tree with nvcc.

Each translation unit is compiled for sm_103a only, in parallel, then linked
into one shared library with the CUDA runtime linked statically.  A rebuild
happens only when a source or header is newer than the library.  Beside it,
g++ builds _binding.so (csrc/binding.cpp, a CPython module against torch's
headers): the Python side of the decode step's calls.

``build(timeline=True)`` builds the same sources with -DPKV_TIMELINE into
libpkv_timeline.so: the attention kernels then stamp %globaltimer at fixed
points into a buffer that ``timeline.py`` reads.  Nothing else loads it.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libpkv.so")
OBJDIR = os.path.join(PKG, "_build")
BINDING = os.path.join(PKG, "_binding.so")
BINDING_ABI = os.path.join(OBJDIR, "binding.abi")   # what it was built for
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
LIB_TIMELINE = os.path.join(PKG, "libpkv_timeline.so")
OBJDIR_TIMELINE = os.path.join(PKG, "_build_timeline")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def stale(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(d) > t for d in _deps())


def _binding_abi() -> str:
    """What _binding.so is compiled for besides its sources: this Python and this torch."""
    import platform
    import sysconfig
    import torch
    return "\n".join((sysconfig.get_config_var("SOABI") or "", platform.machine(), torch.__version__,
                      str(int(torch._C._GLIBCXX_USE_CXX11_ABI)))) + "\n"


def binding_fits() -> bool:
    """Whether the _binding.so that is there was built for this Python and this torch."""
    try:
        with open(BINDING_ABI) as f:
            return os.path.exists(BINDING) and f.read() == _binding_abi()
    except OSError:
        return False


def build_binding(force: bool = False) -> str:
    """_binding.so: reads torch tensors and calls libpkv.so, which it loads when told to.  Rebuilt when a
    source is newer, and when it was built for another Python or torch."""
    newest = max(os.path.getmtime(f) for f in (BINDING_SRC, os.path.join(INCLUDE, "pkv.h"), os.path.abspath(__file__)))
    if not force and binding_fits() and os.path.getmtime(BINDING) >= newest:
        return BINDING
    import sysconfig
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    tmp = BINDING + f".tmp.{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
           "-I", os.path.join(root, "include"), "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-I", os.path.join(cuda, "include"), "-I", sysconfig.get_paths()["include"], BINDING_SRC, "-o", tmp,
           "-L", os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {BINDING_SRC}:\n{r.stdout}\n{r.stderr}")
    os.makedirs(os.path.dirname(BINDING_ABI), exist_ok=True)
    if os.path.exists(BINDING_ABI):
        os.remove(BINDING_ABI)   # none while the two files could disagree
    os.replace(tmp, BINDING)
    with open(BINDING_ABI + f".tmp.{os.getpid()}", "w") as f:
        f.write(_binding_abi())
    os.replace(f.name, BINDING_ABI)
    return BINDING


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False, timeline: bool = False) -> str:
    lib, objdir = (LIB_TIMELINE, OBJDIR_TIMELINE) if timeline else (LIB, OBJDIR)
    if not force and not stale(lib):
        build_binding()
        return lib
    nvcc = _nvcc()
    os.makedirs(objdir, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_info else []
    if timeline:
        extra += ["-DPKV_TIMELINE"]

    def compile_one(src):
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        binding = ex.submit(build_binding, force)
        results = list(ex.map(compile_one, srcs))
        binding.result()
    if verbose or ptxas_info:
        for (_, log), src in zip(results, srcs):
            if log.strip():
                print(f"== {os.path.basename(src)}\n{log}", file=sys.stderr)
    objs = [o for o, _ in results]
    tmp = lib + f".tmp.{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv)
    print(LIB)
