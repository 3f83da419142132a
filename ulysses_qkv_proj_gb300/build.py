"""Build libqnre.so in-tree with nvcc for sm_103a.

    python -m ulysses_qkv_proj_gb300.build            # libqnre.so
    python -m ulysses_qkv_proj_gb300.build --debug    # libqnre_debug.so: bounds-checked accesses

Compiles every csrc/*.cu in parallel, then links the shared library next to
this file.  Only nvcc and the CUDA runtime (linked statically) are needed; the
driver entry point for TMA descriptors is looked up at run time, so the library
also loads on a machine without a GPU driver.
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
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(HERE, "libqnre.so")
MARSHAL_PATH = os.path.join(HERE, "_marshal.so")
DEBUG_BUILD_DIR = os.path.join(HERE, "_build_debug")
DEBUG_LIB_PATH = os.path.join(HERE, "libqnre_debug.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              f"-I{INCLUDE}", "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def build_marshal() -> str:
    """Compile _marshal.so (csrc/marshal.cpp), the binding's native reads of torch tensors.  Returns its path, or
    "" where torch's or Python's headers are missing or g++ does not take them: the binding then reads tensors in
    Python.  A failure is printed, and no older _marshal.so stays behind it."""
    try:
        import torch
        from torch.utils import cpp_extension
    except ImportError:
        return ""
    includes = [sysconfig.get_paths()["include"], *cpp_extension.include_paths()]
    if not os.path.exists(os.path.join(includes[0], "Python.h")) or shutil.which("g++") is None:
        return ""
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = MARSHAL_PATH + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[f"-I{i}" for i in includes], "-w", os.path.join(CSRC, "marshal.cpp"), "-o", tmp, f"-L{libs}",
           "-ltorch_python", "-ltorch_cpu", "-lc10", f"-Wl,-rpath,{libs}"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(f"g++ failed on marshal.cpp, the binding will read tensors in Python:\n{res.stdout}\n{res.stderr}\n")
        for path in (tmp, MARSHAL_PATH):
            if os.path.exists(path):
                os.remove(path)
        return ""
    os.replace(tmp, MARSHAL_PATH)
    return MARSHAL_PATH


def build(verbose: bool = False, ptxas_info: bool = False, debug_bounds: bool = False) -> str:
    """Compile and link the library; `debug_bounds` builds libqnre_debug.so, whose
    kernels check every load and store against its buffer's byte range and skip
    (and count) any access outside it."""
    nvcc = _nvcc()
    build_dir = DEBUG_BUILD_DIR if debug_bounds else BUILD_DIR
    lib_path = DEBUG_LIB_PATH if debug_bounds else LIB_PATH
    defines = ["-DQNRE_DEBUG_BOUNDS=1"] if debug_bounds else []
    os.makedirs(build_dir, exist_ok=True)
    srcs = sources()

    def compile_one(src: str) -> str:
        obj = os.path.join(build_dir, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *defines, "-c", src, "-o", obj]
        if ptxas_info:
            cmd += ["-Xptxas", "-v"]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{res.stdout}\n{res.stderr}")
        if verbose or ptxas_info:
            sys.stdout.write(res.stdout + res.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(srcs) + 1) as ex:
        marshal = None if debug_bounds else ex.submit(build_marshal)
        objs = list(ex.map(compile_one, srcs))
        if marshal is not None:
            marshal.result()
    tmp = lib_path + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, lib_path)
    return lib_path


if __name__ == "__main__":
    print(build(verbose=True, ptxas_info="-v" in sys.argv, debug_bounds="--debug" in sys.argv))
