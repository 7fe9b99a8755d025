"""Build the CUDA library ``libmoe_gb300.so`` in-tree (sm_103a only).

Each ``csrc/*.cu`` file is compiled in parallel with nvcc into ``_build/``
and linked into ``token_dispatch_grouped_moe_gb300/libmoe_gb300.so``. No
cmake, no torch extension machinery: the library is a plain C-ABI shared
object loaded with ctypes. ``csrc/torch_binding.cpp``, the Python calls of the
8-bit operators, is one g++ command against the installed PyTorch's headers
(``_binding.so``, linked to the library beside it).

    python -m token_dispatch_grouped_moe_gb300.build [--force]
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libmoe_gb300.so")
BINDING = os.path.join(PKG, "_binding.so")
SOURCES = ["route.cu", "route_tc.cu", "permute.cu", "permute_static.cu", "grouped_gemm.cu", "combine.cu", "api.cu",
           "selftest.cu", "fp8_gemm.cu", "fp8_quant.cu", "api_fp8.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC", *ARCH]


def nvcc() -> str:
    exe = shutil.which("nvcc")
    if exe:
        return exe
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found: set CUDA_HOME or put nvcc on PATH")


def _deps(src: str) -> list[str]:
    hdrs = [os.path.join(CSRC, h) for h in os.listdir(CSRC) if h.endswith((".cuh", ".h"))]
    hdrs.append(os.path.join(ROOT, "include", "moe.h"))
    return [src, *hdrs]


def _stale(out: str, deps: list[str]) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps if os.path.exists(d))


def _compile(src_name: str, force: bool) -> str:
    src = os.path.join(CSRC, src_name)
    obj = os.path.join(BUILD, src_name.replace(".cu", ".o"))
    if force or _stale(obj, _deps(src)):
        cmd = [nvcc(), *NVCC_FLAGS, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src_name}:\n{r.stdout}\n{r.stderr}")
    return obj


def _run(cmd: list[str], what: str) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _torch_dir() -> str:
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        raise RuntimeError("PyTorch is not installed: the Python binding needs its headers")
    return list(spec.submodule_search_locations)[0]


def _compile_binding(force: bool) -> str:
    src = os.path.join(CSRC, "torch_binding.cpp")
    obj = os.path.join(BUILD, "torch_binding.o")
    if force or _stale(obj, [src, os.path.join(ROOT, "include", "moe.h")]):
        inc = os.path.join(_torch_dir(), "include")
        cuda = os.path.dirname(os.path.dirname(nvcc()))
        dirs = [inc, os.path.join(inc, "torch", "csrc", "api", "include"), os.path.join(cuda, "include"),
                sysconfig.get_paths()["include"]]
        _run(["g++", "-std=c++17", "-O2", "-fPIC", "-fvisibility=hidden", *(f"-I{d}" for d in dirs), "-c", src, "-o",
              obj], "g++ for torch_binding.cpp")
    return obj


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_compile_binding, force)
        objs = list(ex.map(lambda s: _compile(s, force), SOURCES))
        binding_obj = binding.result()
    if force or _stale(LIB, objs):
        tmp = LIB + ".tmp"
        cmd = [nvcc(), "-shared", *ARCH, "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    if force or _stale(BINDING, [binding_obj]):
        tmp = BINDING + ".tmp"
        torch_lib = os.path.join(_torch_dir(), "lib")
        _run(["g++", "-shared", "-o", tmp, binding_obj, f"-L{PKG}", "-l:libmoe_gb300.so", "-Wl,-rpath,$ORIGIN",
              f"-L{torch_lib}", f"-Wl,-rpath,{torch_lib}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"],
             "link of the Python binding")
        os.replace(tmp, BINDING)
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
