"""Build libw4moe.so in-tree with nvcc for sm_103a (one -gencode, parallel TUs), and the
module beside it that calls it with torch tensors."""
from __future__ import annotations

import concurrent.futures as cf
import importlib.metadata
import importlib.util
import os
import re
import shutil
import subprocess
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libw4moe.so")
SOURCES = ["api.cu", "quantize.cu", "route_align.cu", "combine.cu", "grouped_gemm.cu",
           "static_scratch.cu", "rmsnorm.cu", "sampler.cu", "dense_gemm.cu",
           "few.cu", "kv.cu", "attention.cu", "rope.cu",
           "linear_few.cu", "linear_few_wide.cu"]
HEADERS = ["launch.h", "ptx.cuh", "korder.cuh", "combine_fold.cuh", "checks.cuh",
           "route_token.cuh", "attention_plan.cuh", "strides.h"]
CALLS_SOURCE = os.path.join(CSRC, "calls.cpp")
CALLS_HEADERS = [os.path.join(CSRC, "strides.h")]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA library cannot be built")


def calls_path() -> str:
    """The module of csrc/calls.cpp: one for each version of torch, whose headers it takes."""
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:        # torch from a folder of its own
        from torch import __version__ as version
    version = re.sub(r"\W", "_", version)
    return os.path.join(BUILD, f"w4_calls_torch_{version}.so")


def calls_lack() -> str | None:
    """What the module needs and this machine lacks; the library needs none of it."""
    if importlib.util.find_spec("torch") is None:
        return "torch"
    if not shutil.which("g++"):
        return "g++"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python's headers"
    return None


def _stale(target: str, sources: list) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    deps = sources + [os.path.join(ROOT, "include", "w4moe.h"), os.path.abspath(__file__)]
    return any(os.path.getmtime(p) > t for p in deps)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile every translation unit and link the shared library, and the module beside
    it where this machine has what that needs; returns the library's path."""
    lacking = calls_lack()
    if lacking:
        warnings.warn(f"no {lacking}: only the library is built, not the module of the calls that "
                      "need it", stacklevel=2)
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        calls = None
        if not lacking and (force or _stale(calls_path(), [CALLS_SOURCE, *CALLS_HEADERS])):
            calls = ex.submit(_compile_calls)
        if force or ptxas_info or _stale(LIB, [os.path.join(CSRC, f) for f in SOURCES + HEADERS]):
            _compile(BUILD, LIB, [], verbose, ptxas_info)
        if calls:
            calls.result()
    return LIB


def build_checked(out_dir: str) -> str:
    """The library with W4_CHECK_BOUNDS (every data-dependent global store
    range-checked; a failed check sets W4_DEV_OUT_OF_BOUNDS and skips the
    store), built into out_dir for the tests; returns its path."""
    return _compile(out_dir, os.path.join(out_dir, "libw4moe_checked.so"), ["-DW4_CHECK_BOUNDS"],
                    False, False)


def _compile_calls() -> None:
    gxx = shutil.which("g++")
    os.makedirs(BUILD, exist_ok=True)
    torch = list(importlib.util.find_spec("torch").submodule_search_locations)[0]
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    includes = [os.path.join(torch, "include"), os.path.join(torch, "include/torch/csrc/api/include"),
                sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    libs, out = os.path.join(torch, "lib"), calls_path()
    tmp = out + f".tmp{os.getpid()}"
    cmd = [gxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           *[x for i in includes for x in ("-isystem", i)], CALLS_SOURCE, "-o", tmp, "-L", libs,
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda",
           f"-Wl,-rpath,{libs}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {CALLS_SOURCE}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)


def _compile(build_dir: str, lib: str, defines: list, verbose: bool, ptxas_info: bool) -> str:
    os.makedirs(build_dir, exist_ok=True)
    nvcc = _nvcc()
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                    "-I", os.path.join(ROOT, "include"), "--expt-relaxed-constexpr", *defines]
    if ptxas_info:
        flags += ["-Xptxas", "-v"]

    def compile_one(src: str) -> tuple[str, str]:
        obj = os.path.join(build_dir, src.replace(".cu", ".o"))
        cmd = [nvcc, *flags, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stdout + r.stderr

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    if verbose or ptxas_info:
        for _, log in results:
            if log.strip():
                print(log)
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *[o for o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    import sys
    print(build(force=True, verbose=True, ptxas_info="-v" in sys.argv))
