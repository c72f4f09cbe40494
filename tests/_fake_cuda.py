"""The library's host code (include/lmoe_ffn.h) linked against a stand-in for
the CUDA runtime: argument checks, launch sequences and error paths that need
a second device or a failing call run on the CPU."""
import ctypes
import functools
import itertools
import os
import shutil
import subprocess

from tests._harness import built_library

HERE = os.path.dirname(os.path.abspath(__file__))
OBJECTS = ("ffn_api", "ffn_gemm", "ffn_split", "ffn_skinny", "ffn_mx", "ffn_mx_skinny", "rms_norm", "dense_gemm")
_copies = itertools.count()


@functools.lru_cache(maxsize=1)
def _linked(out_dir: str) -> str:
    lib_dir = os.path.dirname(built_library())
    if not all(os.path.exists(os.path.join(lib_dir, o + ".o")) for o in OBJECTS):
        from latent_mixture_experts_gb300 import build
        build.build(force=True)
    so = os.path.join(out_dir, "libfake.so")
    nvcc = shutil.which(os.environ.get("NVCC", "nvcc"))
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    # -Bsymbolic: a CUDA runtime that the process has loaded does not take the stand-in's place
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wl,-Bsymbolic", "-I", include,
                    os.path.join(HERE, "_fake_cuda.cpp"),
                    *(os.path.join(lib_dir, o + ".o") for o in OBJECTS), "-o", so], check=True)
    return so


def load(tmp_factory):
    """A library of its own: nothing kept from another test's calls."""
    from latent_mixture_experts_gb300 import binding as b
    d = _directory(tmp_factory)
    path = os.path.join(d, f"libfake{next(_copies)}.so")
    shutil.copy(_linked(d), path)
    lib = ctypes.CDLL(path)
    real = b.load_library()
    for name in b.EXPORTS:
        if hasattr(lib, name):
            f, g = getattr(lib, name), getattr(real, name)
            f.restype, f.argtypes = g.restype, g.argtypes
    return lib


_dirs = {}


def _directory(tmp_factory) -> str:
    return _dirs.setdefault("d", str(tmp_factory.mktemp("fake_cuda")))
