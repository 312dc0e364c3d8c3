"""Builds the in-tree CUDA library libmoe_w4a16.so for sm_103a with nvcc.

Every .cu under csrc/ is compiled in parallel to an object, then linked into
one shared library (static CUDA runtime, C ABI of include/moe_w4a16.h).
csrc/block_binding.cpp becomes the Python module _lib/_block.so beside it
(the tensor checks of the block operators; links against torch and the
library).
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT_DIR = os.path.join(PKG, "_lib")
LIB = os.path.join(OUT_DIR, "libmoe_w4a16.so")
BINDING_SRC = os.path.join(CSRC, "block_binding.cpp")
BINDING = os.path.join(OUT_DIR, "_block.so")
STAMP = os.path.join(OUT_DIR, "_block.txt")   # what the binding was built against
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        [os.path.join(ROOT, "include", "moe_w4a16.h"), __file__]


def _newer(target, deps) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(p) <= os.path.getmtime(target) for p in deps)


def _built_against() -> str:
    """The versions that the binding's ABI depends on."""
    import sys

    import torch
    return f"torch {torch.__version__}, CXX11 ABI {int(torch._C._GLIBCXX_USE_CXX11_ABI)}, python {sys.version.split()[0]}"


def _stamped() -> bool:
    try:
        with open(STAMP) as f:
            return f.read() == _built_against()
    except OSError:
        return False


def up_to_date() -> bool:
    return _newer(LIB, _deps()) and _newer(BINDING, [BINDING_SRC, LIB, __file__]) and _stamped()


def _compile_binding() -> str:
    """block_binding.cpp -> object (linked once the library is there)."""
    import sysconfig

    import torch
    tdir = os.path.dirname(torch.__file__)
    obj = os.path.join(OUT_DIR, "block_binding.o")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    inc = [os.path.join(tdir, "include"), os.path.join(tdir, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include"), os.path.join(ROOT, "include")]
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={abi}", *[f"-I{d}" for d in inc], "-c", BINDING_SRC, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {BINDING_SRC}:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_binding(obj: str) -> None:
    import torch
    tlib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = [shutil.which("g++") or "g++", "-shared", "-o", BINDING + ".tmp", obj, f"-L{tlib}", "-ltorch_python",
           "-ltorch_cpu", "-lc10_cuda", "-lc10", f"-L{OUT_DIR}", "-l:libmoe_w4a16.so", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(BINDING + ".tmp", BINDING)
    with open(STAMP, "w") as f:
        f.write(_built_against())
    os.remove(obj)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    cc = nvcc()
    objs = []

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *ARCH, *FLAGS, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with concurrent.futures.ThreadPoolExecutor(max_workers=min(12, os.cpu_count() or 1)) as ex:
        binding = ex.submit(_compile_binding)
        for obj, log in ex.map(compile_one, _sources()):
            objs.append(obj)
            if verbose and log:
                print(log)
        binding_obj = binding.result()
    tmp = LIB + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs, "-lcuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    for o in objs:
        os.remove(o)
    _link_binding(binding_obj)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
