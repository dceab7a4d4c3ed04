"""Build libmk.so in-tree with nvcc for sm_103a (GB300), and the Python module
_mktorch.so that calls it on torch tensors with the host compiler.

Each translation unit compiles in parallel, then nvcc links the shared
library next to this file.  Nothing is installed anywhere else.
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmk.so")
MODULE = os.path.join(HERE, "_mktorch.so")
SOURCES = ["mk_kernels_d128.cu", "mk_kernels_hidden1024.cu", "mk_kernels_hidden2048.cu", "mk_kernels_d64.cu",
           "mk_host.cu", "mk_embed.cu", "mk_prefill.cu", "mk_gemm.cu", "mk_pfattn.cu",
           "mk_paged.cu", "mk_q4.cu", "mk_q4_bf16.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cand = os.path.join(cuda, "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("command failed: %s\n%s%s" % (" ".join(cmd), r.stdout, r.stderr))
    return r.stdout + r.stderr


def _torch_dir() -> str:
    import torch
    return os.path.dirname(torch.__file__)


def _compile_module(obj: str) -> str:
    inc = os.path.join(_torch_dir(), "include")
    cuda = os.path.dirname(os.path.dirname(_nvcc())) or "/usr/local/cuda"
    dirs = [inc, os.path.join(inc, "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    return _run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", *["-I" + d for d in dirs], "-c",
                 os.path.join(CSRC, "mk_torch.cpp"), "-o", obj])


def _link_module(obj: str) -> None:
    lib = os.path.join(_torch_dir(), "lib")
    tmp = MODULE + ".tmp"
    _run(["g++", "-shared", "-o", tmp, obj, "-L" + HERE, "-l:libmk.so", "-Wl,-rpath,$ORIGIN", "-L" + lib, "-Wl,-rpath," + lib,
          "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10_cuda", "-lc10"])
    os.replace(tmp, MODULE)


def build(verbose: bool = False, ptxas_info: bool = False, module: bool = True) -> str:
    """Compile and link libmk.so and, unless ``module`` is false, _mktorch.so;
    returns libmk.so's path.  libmk.so needs nvcc alone and is there even if
    _mktorch.so, which needs torch, Python's headers and g++, raises."""
    os.makedirs(OUT_DIR, exist_ok=True)
    nvcc = _nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []
    objs = [os.path.join(OUT_DIR, s.replace(".cu", ".o")) for s in SOURCES]

    def one(i):
        return _run([nvcc, *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, SOURCES[i]), "-o", objs[i]])

    module_obj = os.path.join(OUT_DIR, "mk_torch.o")
    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        made = ex.submit(_compile_module, module_obj) if module else None
        logs = list(ex.map(one, range(len(SOURCES))))
        tmp = LIB + ".tmp"
        _run([nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"])
        os.replace(tmp, LIB)
        if module:
            try:
                made.result()
                _link_module(module_obj)
            except (ImportError, OSError, RuntimeError) as e:
                if os.path.exists(MODULE):               # one of an earlier build may expect another libmk.so
                    os.remove(MODULE)
                raise RuntimeError("%s is built, _mktorch.so (the serving operators on torch tensors) is not: %s" % (LIB, e)) from e
    if verbose:
        for s, log in zip(SOURCES, logs):
            if log.strip():
                print("== %s\n%s" % (s, log))
    return LIB


if __name__ == "__main__":
    build(verbose=True, ptxas_info="-v" in sys.argv, module="--library" not in sys.argv)   # --library: libmk.so alone
    print(LIB)
