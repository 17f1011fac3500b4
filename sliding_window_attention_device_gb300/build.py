"""Builds libbdattn.so (the CUDA kernels behind include/bdattn.h) in-tree with nvcc.

Every translation unit is compiled for sm_103a only, in parallel, then linked
into one shared library next to this file; so is _calls, the part of the Python
binding that small calls go through (g++, against the Python and torch that are
installed, of which its file is named). Run as ``python -m
sliding_window_attention_device_gb300.build``.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libbdattn.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", f"-I{os.path.join(ROOT, 'include')}"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libbdattn.so")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(ROOT, "include", "*.h")))


def _calls_source() -> str:
    return os.path.join(CSRC, "calls.cpp")


def calls_path() -> str:
    """The file of _calls for this Python and this torch: it inlines structs of both, so another version of either
    looks for, and builds, a file of its own."""
    import torch
    tag = f"{sysconfig.get_config_var('SOABI')}.torch-{torch.__version__}"
    return os.path.join(PKG, f"_calls.{re.sub(r'[^A-Za-z0-9_.+-]', '_', tag)}.so")


def _older(path: str, sources) -> bool:
    return not os.path.exists(path) or any(os.path.getmtime(p) > os.path.getmtime(path) for p in sources)


def library_stale() -> bool:
    return _older(LIB, _sources() + _headers() + [__file__])


def calls_stale() -> bool:
    return _older(calls_path(), [_calls_source(), os.path.join(ROOT, "include", "bdattn.h"), __file__])


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    return r.stdout + r.stderr


def _calls_includes():
    """The folders of the headers that _calls is compiled against, each behind the name of one of its files; none
    where torch is not installed."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return []
    torch = os.path.join(list(spec.submodule_search_locations)[0], "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    return [("bdattn.h", os.path.join(ROOT, "include")), ("Python.h", sysconfig.get_paths()["include"]),
            ("cuda_runtime.h", cuda), ("ATen/core/Tensor.h", torch),
            ("torch/all.h", os.path.join(torch, "torch", "csrc", "api", "include"))]


def calls_lack() -> str:
    """What _calls needs to be built and is not here, or an empty text. The library needs none of it."""
    if shutil.which("g++") is None:
        return "g++"
    includes = _calls_includes()
    if not includes:
        return "torch"
    return ", ".join(os.path.join(d, f) for f, d in includes if not os.path.isfile(os.path.join(d, f)))


def _compile_calls() -> str:
    obj = os.path.join(BUILD_DIR, "calls.o")
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", *(f"-I{d}" for _, d in _calls_includes()), "-c",
          _calls_source(), "-o", obj], "g++ for calls.cpp")
    return obj


def _link_calls(obj: str):
    lib = os.path.join(list(importlib.util.find_spec("torch").submodule_search_locations)[0], "lib")
    path = calls_path()
    tmp = path + f".tmp{os.getpid()}"
    _run(["g++", "-shared", "-o", tmp, obj, f"-L{PKG}", "-l:libbdattn.so", f"-L{lib}", "-lc10", "-lc10_cuda",
          "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN"], "link of _calls")
    os.replace(tmp, path)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile what is stale and return the path of libbdattn.so. _calls is left out, with a note, where what it alone
    needs is not installed."""
    library = force or library_stale()
    calls = importlib.util.find_spec("torch") is None or force or calls_stale()
    if calls and (lack := calls_lack()):
        print(f"_calls is left out: {lack} not found", file=sys.stderr)
        calls = False
    if not library and not calls:
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        out = _run([nvcc, *ARCH, *FLAGS, "-c", src, "-o", obj], f"nvcc for {src}")
        if verbose:
            sys.stdout.write(out)
        return obj

    with cf.ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        calls_obj = ex.submit(_compile_calls) if calls else None
        if library:
            objs = list(ex.map(compile_one, _sources()))
            tmp = LIB + f".tmp{os.getpid()}"
            _run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], "link of libbdattn.so")
            os.replace(tmp, LIB)
        if calls:
            _link_calls(calls_obj.result())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
