"""Builds the in-tree shared library ``_lib/libflce.so`` with nvcc for sm_103a,
and ``_lib/_flce_torch.so``, the Python module over it.

Each .cu file is compiled to an object in parallel, then linked with the
static CUDA runtime (the library needs no libcudart at load time and finds
the CUDA driver entry points it uses at run time).  The module is plain C++
against the installed torch's headers; without torch only the library is built
(``python lm_head_linear_flce_gb300/_build.py``).
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
OUT_DIR = os.path.join(PKG, "_lib")
LIB = os.path.join(OUT_DIR, "libflce.so")
MODULE = os.path.join(OUT_DIR, "_flce_torch.so")
SOURCES = ["flce_api.cu", "flce_simt.cu", "flce_gemm.cu", "flce_noalloc.cu",
           "flce_ops.cu", "flce_norm.cu", "flce_fp8.cu", "flce_process.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libflce.so")


def _run(cmd: list[str], what: str) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _compile_module(obj: str) -> None:
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    dirs = [inc, os.path.join(inc, "torch", "csrc", "api", "include"),
            sysconfig.get_paths()["include"], cuda]
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    _run(["g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={abi}",
          *(f"-I{d}" for d in dirs), "-c", os.path.join(CSRC, "flce_torch.cpp"), "-o", obj],
         "g++ on flce_torch.cpp")


def _link_module(obj: str) -> None:
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = MODULE + ".tmp"
    _run(["g++", "-shared", obj, "-o", tmp, f"-L{OUT_DIR}", "-lflce", "-Wl,-rpath,$ORIGIN",
          f"-L{lib}", f"-Wl,-rpath,{lib}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"],
         "linking _flce_torch.so")
    os.replace(tmp, MODULE)


def _compile(src: str, obj: str, extra: list[str]) -> None:
    cmd = [nvcc(), *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")


def build(verbose: bool = False, extra: list[str] | None = None) -> str:
    extra = list(extra or [])
    os.makedirs(OUT_DIR, exist_ok=True)
    objs = [os.path.join(OUT_DIR, s.replace(".cu", ".o")) for s in SOURCES]
    module_obj = os.path.join(OUT_DIR, "flce_torch.o")
    try:
        import torch  # noqa: F401
        no_torch = None
    except ImportError as e:
        no_torch = e
    with concurrent.futures.ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        futs = [ex.submit(_compile, s, o, extra) for s, o in zip(SOURCES, objs)]
        module = None if no_torch else ex.submit(_compile_module, module_obj)
        for f in futs:
            f.result()
        # the library first: it needs nothing of the module's
        tmp = LIB + ".tmp"
        cmd = [nvcc(), *ARCH, "-shared", "-Xcompiler", "-fPIC", "-cudart", "static", *objs,
               "-o", tmp]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
        try:
            if module is not None:
                module.result()
                _link_module(module_obj)
        except Exception:
            _remove_module()
            raise
    if no_torch:
        _remove_module()
        print(f"built {LIB} without the Python module over it: torch cannot be imported "
              f"({no_torch})", file=sys.stderr)
    if verbose:
        print("built", LIB)
    return LIB


def _remove_module() -> None:
    """No module is better than one of another library's: its calls then say so."""
    if os.path.exists(MODULE):
        os.remove(MODULE)


if __name__ == "__main__":
    build(verbose=True)
