"""Build the in-tree CUDA library ``libpagedserve.so`` for sm_103a with nvcc, and the Python
module ``_native`` that calls it with the host compiler.

Each ``csrc/*.cu`` file compiles in parallel to an object under ``_build/`` at the
repository root; the objects link into ``paged_kv_attention_18_gb300/libpagedserve.so``
with the CUDA runtime linked statically. Objects are rebuilt when a source or header
is newer. The library needs nvcc alone: where torch is not installed the Python module is left
out, and where it does not compile (no host C++ compiler, no Python headers) the error comes
once the library is in place.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import shutil
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libpagedserve.so")
NATIVE = os.path.join(PKG, "_native.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         f"-I{INCLUDE}", f"-I{CSRC}"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build the library")


def _run(cmd: list[str], what: str, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        print(r.stdout + r.stderr, flush=True)


def _native_object(verbose: bool) -> str:
    """The Python module's object, by the torch it is compiled against."""
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    src = os.path.join(CSRC, "py_native.cpp")
    obj = os.path.join(BUILD, f"py_native.{torch.__version__}.o")
    if not os.path.exists(obj) or os.path.getmtime(obj) < max(os.path.getmtime(src),
                                                              _newest_header()):
        cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
        abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
        _run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC",
              f"-D_GLIBCXX_USE_CXX11_ABI={abi}", f"-I{INCLUDE}",
              f"-I{sysconfig.get_paths()['include']}", f"-I{inc}",
              f"-I{os.path.join(inc, 'torch', 'csrc', 'api', 'include')}", f"-I{cuda}", "-c", src,
              "-o", obj], f"compiling {src}", verbose)
    return obj


def _link_native(obj: str, verbose: bool) -> None:
    import torch
    stamp = os.path.join(BUILD, "native.stamp")  # the object the module was linked from
    linked = open(stamp).read() if os.path.exists(stamp) else ""
    if os.path.exists(NATIVE) and linked == obj and \
            os.path.getmtime(NATIVE) >= max(os.path.getmtime(obj), os.path.getmtime(LIB)):
        return
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = NATIVE + ".tmp"
    _run([os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, f"-L{PKG}",
          "-l:libpagedserve.so", f"-L{libs}", "-ltorch_python", "-ltorch", "-ltorch_cpu",
          "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{libs}"],
         "linking the Python module", verbose)
    os.replace(tmp, NATIVE)
    with open(stamp, "w") as f:
        f.write(obj)


def _newest_header() -> float:
    hs = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))
    return max((os.path.getmtime(h) for h in hs), default=0.0)


def build(verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    hdr_time = _newest_header()
    cc = nvcc()
    flags = FLAGS + list(extra_flags or [])

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        if (not os.path.exists(obj) or os.path.getmtime(obj) < max(os.path.getmtime(src), hdr_time)
                or extra_flags):
            cmd = [cc, *ARCH, *flags, "-c", src, "-o", obj]
            if verbose:
                print(" ".join(cmd), flush=True)
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
            if verbose and (r.stdout or r.stderr):
                print(r.stdout + r.stderr, flush=True)
        return obj

    # (the host compiler's one object beside nvcc's)
    with ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        native = ex.submit(_native_object, verbose) if importlib.util.find_spec("torch") else None
        objs = list(ex.map(compile_one, srcs))
    if (not os.path.exists(LIB) or os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs)):
        tmp = LIB + ".tmp"
        _run([cc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs], "nvcc link", verbose)
        os.replace(tmp, LIB)
    if native is not None:
        _link_native(native.result(), verbose)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
