"""Builds libfp8blk.so in-tree with nvcc for sm_103a.

Each .cu translation unit compiles in parallel to an object, then one nvcc
link makes the shared library (static CUDA runtime, so loading it needs no
GPU and no libcudart on the library path). The CUDA driver is reached at run
time through the runtime's entry-point query (for cuTensorMapEncodeTiled), so
the library does not link libcuda either.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libfp8blk.so")
BIND = os.path.join(PKG, "_bind.so")
BUILD = os.path.join(PKG, "_build")
BIND_FOR = os.path.join(BUILD, "bind.for")   # what BIND was compiled against

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return hs


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


class BindError(RuntimeError):
    """The native part of the Python binding could not be compiled; the C library is there."""


def bind_for() -> str:
    """The torch and the interpreter that the native part of the binding is compiled against."""
    import sys

    import torch
    return f"torch {torch.__version__} at {os.path.dirname(torch.__file__)}, python {sys.version}"


def _bind_is_stale() -> bool:
    if _stale(BIND, [os.path.join(CSRC, "bind.cpp"), os.path.join(INCLUDE, "fp8blk.h")]) or not os.path.exists(BIND_FOR):
        return True
    with open(BIND_FOR) as f:
        return f.read() != bind_for()


def bind_command(out: str) -> list[str]:
    """Compiles the native part of the Python binding against the installed torch."""
    import sysconfig

    import torch
    inc, lib = (os.path.join(os.path.dirname(torch.__file__), d) for d in ("include", "lib"))
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    return ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE, "-I", inc,
            "-I", os.path.join(inc, "torch", "csrc", "api", "include"), "-I", sysconfig.get_paths()["include"],
            "-I", os.path.join(cuda, "include"), os.path.join(CSRC, "bind.cpp"), "-o", out,
            "-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", f"-Wl,-rpath,{lib}"]


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compiles what is out of date: the C library, which needs nvcc alone, and, where torch is installed, the native part
    of the Python binding. Where that fails BindError is raised after the library has been linked."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()
    hdrs = _headers()
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in srcs]
    nv = nvcc()

    def compile_one(pair):
        src, obj = pair
        if force or _stale(obj, [src] + hdrs):
            cmd = [nv, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
            if verbose:
                print(" ".join(cmd), flush=True)
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
            if verbose and (r.stdout or r.stderr):
                print(r.stdout, r.stderr, flush=True)
        return obj

    def compile_bind():
        if importlib.util.find_spec("torch") is None:
            return
        try:
            if not force and not _bind_is_stale():
                return
            tmp = BIND + f".tmp{os.getpid()}"
            r = subprocess.run(bind_command(tmp), capture_output=True, text=True)
        except (OSError, ImportError) as e:
            raise BindError(f"bind.cpp was not compiled ({e}); {LIB} does not need it") from e
        if r.returncode != 0:
            raise BindError(f"g++ failed on bind.cpp ({LIB} does not need it):\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, BIND)
        with open(BIND_FOR, "w") as f:
            f.write(bind_for())

    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        bind = ex.submit(compile_bind)
        list(ex.map(compile_one, zip(srcs, objs)))
        if force or _stale(LIB, objs):
            tmp = LIB + f".tmp{os.getpid()}"
            cmd = [nv, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
            os.replace(tmp, LIB)
        bind.result()
    return LIB


if __name__ == "__main__":
    import sys

    try:
        print(build(force="--force" in sys.argv, verbose=True))
    except BindError as e:
        print(LIB)
        print(f"{e}\nwithout it the Python binding has no 4-bit calls and no residual_norm", file=sys.stderr)
