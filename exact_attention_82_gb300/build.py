"""Build the sm_103a shared library in-tree with nvcc (no cmake, no torch
extension machinery): each .cu is compiled in parallel, then linked with the
static CUDA runtime into ``_build/libfa_gb300.so``.  The driver's tensor-map
encoder is looked up at run time, so the library does not link libcuda.  The
paged cache's calls for torch tensors are a small CPython extension beside it
(``fa_binding.cpp``, compiled with g++ against torch's headers).  Only those
calls need it: the library is built and loaded without torch or g++.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(HERE, "_build")
LIB_NAME = "libfa_gb300.so"
LIB_PATH = os.path.join(OUT_DIR, LIB_NAME)
BINDING_SOURCE = "fa_binding.cpp"
BINDING_PATH = os.path.join(OUT_DIR, "fa_binding.so")

SOURCES = ["fa_fwd_kernel.cu", "fa_splitkv.cu", "fa_bwd.cu", "fa_kv_cache.cu", "fa_page_select.cu",
           "fa_paged.cu", "fa_api.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", INCLUDE]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")


def _gxx() -> str:
    path = shutil.which("g++")
    if path is None:
        raise RuntimeError("g++ not found: the paged cache's calls on tensors need it (their *_raw forms do not)")
    return path


def _inputs():
    files = [os.path.join(CSRC, s) for s in SOURCES]
    files += [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    files += [os.path.join(INCLUDE, "fa.h"), os.path.abspath(__file__)]
    return files


def _binding_inputs():
    return [os.path.join(CSRC, BINDING_SOURCE), os.path.join(INCLUDE, "fa.h"), os.path.abspath(__file__)]


def _binding_key() -> str:
    """What the binding's binary interface depends on: torch's build and Python's."""
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        return f"{sysconfig.get_config_var('EXT_SUFFIX')}\n{_torch_dir()}\n{f.read()}"


def _binding_key_was() -> str | None:
    try:
        with open(BINDING_PATH + ".key") as f:
            return f.read()
    except OSError:
        return None


def _newer(path: str, inputs) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(f) <= os.path.getmtime(path) for f in inputs)


def up_to_date() -> bool:
    return _newer(LIB_PATH, _inputs())


def binding_up_to_date() -> bool:
    return _newer(BINDING_PATH, _binding_inputs()) and _binding_key_was() == _binding_key()


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile and link the library; returns its path."""
    if not force and up_to_date():
        return LIB_PATH
    os.makedirs(OUT_DIR, exist_ok=True)
    cc = nvcc()
    # Objects lie in a folder of this build's own: another process may build at the same time.
    with tempfile.TemporaryDirectory(dir=OUT_DIR) as work:

        def compile_one(src):
            obj = os.path.join(work, os.path.splitext(src)[0] + ".o")
            _run([cc, *ARCH, *FLAGS, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj], f"nvcc on {src}", verbose)
            return obj

        with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
            objs = list(ex.map(compile_one, SOURCES))
        tmp = os.path.join(work, LIB_NAME)
        _run([cc, *ARCH, "-shared", "-Xlinker", f"-soname={LIB_NAME}", "-o", tmp, *objs, "-lcudart_static", "-ldl", "-lpthread", "-lrt"],
             "linking the library", verbose)
        os.replace(tmp, LIB_PATH)
    return LIB_PATH


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """Compile and link the calls on torch tensors, and the library that they need; returns their path."""
    if not force and binding_up_to_date() and up_to_date():
        return BINDING_PATH
    os.makedirs(OUT_DIR, exist_ok=True)
    with tempfile.TemporaryDirectory(dir=OUT_DIR) as work:
        with cf.ThreadPoolExecutor(max_workers=2) as ex:
            lib = ex.submit(build, force, verbose)
            binding = ex.submit(_compile_binding, work, verbose)
            lib.result()  # whatever becomes of the binding, the library is in its place
            _link_binding(binding.result(), work, verbose)
    return BINDING_PATH


def _torch_dir() -> str:
    import importlib.util

    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("torch is not installed: the paged cache's calls on tensors need it (their *_raw forms do not)")
    return os.path.dirname(spec.origin)


def _run(cmd, what: str, verbose: bool = False):
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        print(r.stdout + r.stderr, file=sys.stderr)


def _compile_binding(work: str, verbose: bool) -> str:
    obj = os.path.join(work, "fa_binding.o")
    inc = os.path.join(_torch_dir(), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    _run([_gxx(), "-O2", "-std=c++17", "-fPIC", "-I", sysconfig.get_path("include"), "-isystem", inc,
          "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", cuda, "-c",
          os.path.join(CSRC, BINDING_SOURCE), "-o", obj], f"g++ on {BINDING_SOURCE}", verbose)
    return obj


def _link_binding(obj: str, work: str, verbose: bool) -> None:
    tmp = os.path.join(work, "fa_binding.so")
    libs = os.path.join(_torch_dir(), "lib")
    _run([_gxx(), "-shared", "-o", tmp, obj, LIB_PATH, "-L", libs, "-ltorch_python", "-lc10_cuda", "-lc10",
          "-ltorch_cpu", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{libs}"], "linking the binding", verbose)
    with open(tmp + ".key", "w") as f:
        f.write(_binding_key())
    os.replace(tmp, BINDING_PATH)
    os.replace(tmp + ".key", BINDING_PATH + ".key")


if __name__ == "__main__":
    print(build_binding(force="--force" in sys.argv, verbose="-v" in sys.argv))
