"""Build libqlora.so in-tree for sm_100a with nvcc, its debug build
libqlora_debug.so (-DQLORA_DEBUG_CHECKS: index-range checks in the kernels),
and with g++ the compiled part of the Python binding, module _calls.

    python -m bit_nf4_quantized_21_b200.build        # rebuild when sources changed
    python -m bit_nf4_quantized_21_b200.build -v     # also print ptxas resource usage
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libqlora.so")
LIB_DEBUG = os.path.join(PKG, "libqlora_debug.so")

NVCC_FLAGS = [
    "-O3", "-std=c++17", "-lineinfo",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-Xcompiler", "-fPIC", "-shared",
    "--expt-relaxed-constexpr",
]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(INCLUDE, "*.h")))


def needs_build(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(s) > t for s in _sources())


def build(force: bool = False, verbose: bool = False, debug: bool = False) -> str:
    lib = LIB_DEBUG if debug else LIB
    build_calls(force)
    if not force and not needs_build(lib) and not verbose:
        return lib
    nvcc = os.environ.get("NVCC", "nvcc")
    tmp = lib + f".{os.getpid()}.tmp"
    cmd = [nvcc, *NVCC_FLAGS, *(["-DQLORA_DEBUG_CHECKS"] if debug else []), "-I", INCLUDE, "-I", CSRC,
           "-o", tmp, os.path.join(CSRC, "qlora.cu")]
    if verbose:
        cmd[1:1] = ["-Xptxas", "-v"]
    subprocess.run(cmd, check=True)
    os.replace(tmp, lib)
    return lib


def calls_path() -> str:
    """Where the binding of this interpreter and this torch lies.  Its code depends on the layouts of
    both, so both are in its name: another one's binary is not there to be loaded."""
    import torch
    return os.path.join(PKG, f"_calls.torch-{torch.__version__}{sysconfig.get_config_var('EXT_SUFFIX')}")


def _calls_sources():
    return [os.path.join(CSRC, "calls.cpp"), os.path.join(INCLUDE, "qlora.h")]


def calls_need_build() -> bool:
    path = calls_path()
    return not os.path.exists(path) or any(os.path.getmtime(s) > os.path.getmtime(path) for s in _calls_sources())


def build_calls(force: bool = False) -> str:
    """Module _calls: host code against the headers and libraries of the installed torch."""
    path = calls_path()
    if not force and not calls_need_build():
        return path
    import torch
    torch_dir = os.path.dirname(torch.__file__)
    cuda = os.environ.get("CUDA_HOME") or "/usr/local/cuda"
    include = [INCLUDE, os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include/torch/csrc/api/include"),
               os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    tmp = path + f".{os.getpid()}.tmp"
    # the compiler that nvcc uses too: one that links libstdc++ statically would put a second copy beside torch's
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-Wno-attributes",
                    *(f for d in include for f in ("-isystem", d)), "-o", tmp, _calls_sources()[0],
                    "-L", os.path.join(torch_dir, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", "-ldl"],
                   check=True)
    os.replace(tmp, path)
    return path


if __name__ == "__main__":
    print(build(force=True, verbose="-v" in sys.argv))
    print(build(force=True, debug=True))
