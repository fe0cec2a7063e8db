"""Build libconv2d.so (the C-ABI CUDA library) in-tree for sm_103a.

Translation units are compiled in parallel with nvcc and linked into
conv2d_layer_gb300/_build/libconv2d.so (CUDA runtime linked statically; the
driver API is reached through cudaGetDriverEntryPointByVersion, so libcuda is
not linked). The torch side of ops.py (csrc/binding.cpp) is compiled by the host
compiler into _build/_binding.so; it needs torch's headers and no nvcc.
"""
import concurrent.futures as cf
import importlib.machinery
import importlib.util
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "_build")
LIB = os.path.join(OUT, "libconv2d.so")
SOURCES = ["api.cu", "bn_kernels.cu", "dense.cu", "dense_gemm.cu", "gemm_bf16.cu", "gemm_tf32.cu", "layer_norm.cu", "moe.cu",
           "noalloc.cu", "rms_norm.cu", "rows.cu"]
BINDING = os.path.join(OUT, "_binding.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include")]


def _nvcc():
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != "binding.cpp"] + [os.path.join(ROOT, "include", "conv2d.h")]
    return max(os.path.getmtime(f) for f in files)


def build(force=False, verbose=False, extra=()):
    """Compile the library if it is missing or older than its sources; return its path."""
    os.makedirs(OUT, exist_ok=True)
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= _deps():
        return LIB
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(OUT, src.replace(".cu", ".o"))
        cmd = [nvcc] + ARCH + FLAGS + list(extra) + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, r.stdout, r.stderr))
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [nvcc] + ARCH + ["-shared", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    return LIB


def build_binding(force=False):
    """Compile the binding if it is missing or older than its sources; return its path."""
    os.makedirs(OUT, exist_ok=True)
    deps = max(os.path.getmtime(f) for f in (BINDING_SRC, os.path.join(ROOT, "include", "conv2d.h")))
    if not force and os.path.exists(BINDING) and os.path.getmtime(BINDING) >= deps:
        return BINDING
    import torch

    top = os.path.dirname(torch.__file__)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    inc = [os.path.join(ROOT, "include"), os.path.join(top, "include"),
           os.path.join(top, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include"),
           sysconfig.get_paths()["include"]]
    tmp = BINDING + ".tmp%d" % os.getpid()
    cmd = (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI)] + ["-I" + i for i in inc]
           + [BINDING_SRC, "-o", tmp, "-L" + os.path.join(top, "lib"), "-lc10", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python",
              "-lc10_cuda", "-ldl"])
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("the binding's compilation failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, BINDING)
    return BINDING


def load_binding():
    """The binding as a Python module (torch is imported first: it brings the libraries it is linked to)."""
    import torch  # noqa: F401

    path = build_binding()
    loader = importlib.machinery.ExtensionFileLoader("_binding", path)
    module = importlib.util.module_from_spec(importlib.util.spec_from_file_location("_binding", path, loader=loader))
    loader.exec_module(module)
    return module


if __name__ == "__main__":
    v = "-v" in sys.argv
    extra = ["-Xptxas", "-v"] if "--ptxas" in sys.argv else []
    print(build(force=True, verbose=v or bool(extra), extra=extra))
    print(build_binding(force=True))
