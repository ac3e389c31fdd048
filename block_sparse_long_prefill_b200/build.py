"""Build libmoba.so (the sm_100a CUDA kernels and their C ABI) with nvcc and the compiled
binding of its short calls with the host compiler, both in-tree."""
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libmoba.so")
SOURCES = ["api.cu", "select.cu", "gate.cu", "attn.cu", "merge.cu", "noalloc.cu", "bwd.cu",
           "swa_fwd.cu", "swa_bwd.cu", "rope.cu", "decode.cu"]
HEADERS = ["common.cuh", "params.h", "lists.cuh", "rows.cuh", "swa_tile.cuh"]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "--expt-relaxed-constexpr",
    "-Xcompiler", "-fPIC", "-shared",
]


def binding_path() -> str:
    """The compiled binding of the short calls (binding.cpp).  It is built against one torch and
    one Python; its name says which, so that another finds none instead of a wrong one."""
    import importlib.machinery

    import torch
    return os.path.join(PKG, f"_binding-{torch.__version__}{importlib.machinery.EXTENSION_SUFFIXES[0]}")


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _older(target: str, deps) -> bool:
    return not os.path.exists(target) or any(os.path.getmtime(p) > os.path.getmtime(target) for p in deps)


def _stale() -> bool:
    return _older(LIB, [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [os.path.join(INCLUDE, "moba.h")])


def _build_binding(verbose: bool = False) -> None:
    """Compile the binding against the installed torch; it finds libmoba.so beside itself."""
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    path = binding_path()
    tmp = path + f".tmp{os.getpid()}"
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    cmd = [os.environ.get("CXX") or shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-shared",
           "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE, "-I", sysconfig.get_paths()["include"], "-I", cuda,
           *[f for p in include_paths() for f in ("-isystem", p)],
           os.path.join(CSRC, "binding.cpp"), "-o", tmp, "-L", PKG, "-l:libmoba.so", "-Wl,-rpath,$ORIGIN",
           "-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, path)


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """Compile libmoba.so for sm_100a (cross-compiles without a GPU) and its binding.  Each
    source is compiled to an object file in parallel, then the objects are linked."""
    if force or _stale():
        _build_library(verbose, extra)
    if force or _older(binding_path(), [os.path.join(CSRC, "binding.cpp"), os.path.join(INCLUDE, "moba.h")]):
        _build_binding(verbose)
    return LIB


def _build_library(verbose: bool, extra) -> None:
    from concurrent.futures import ThreadPoolExecutor
    objdir = os.path.join(PKG, "_build")
    os.makedirs(objdir, exist_ok=True)
    compile_flags = [f for f in NVCC_FLAGS if f != "-shared"]

    def compile_one(f):
        obj = os.path.join(objdir, f.replace(".cu", f".{os.getpid()}.o"))
        cmd = [_nvcc(), *compile_flags, *extra, "-I", INCLUDE, "-I", CSRC, "-c",
               os.path.join(CSRC, f), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.check_call(cmd)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [_nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-Xcompiler", "-fPIC",
           *objs, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    for o in objs:
        os.remove(o)
    os.replace(tmp, LIB)


if __name__ == "__main__":
    extra = ["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else []
    print(build(force=True, verbose=True, extra=extra))
