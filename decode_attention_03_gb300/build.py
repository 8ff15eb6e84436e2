"""Build ``libgqa_decode.so`` (the C-ABI library) in-tree with nvcc for sm_103a.

Each ``csrc/*.cu`` translation unit is compiled in parallel to ``_build/*.o``,
then linked into ``decode_attention_03_gb300/libgqa_decode.so`` with the CUDA
runtime linked statically (the library needs only the NVIDIA driver at run
time).  A rebuild happens only when a source or header is newer than the
library.

``csrc/torch_calls.cpp``, the calls that take torch tensors directly, becomes the extension module
``_calls`` beside it (g++, against the installed torch's headers), linked to the library.  Its file carries Python's
tag, it carries the torch version that it was built against, and another torch or Python builds it anew.

``build(checked=True)`` makes the checked library instead,
``libgqa_decode_checked.so`` (objects in ``_build_checked/``): the same sources
compiled with ``GQA_BOUNDS_CHECK=1``, under which the kernels range-check every
computed global- and shared-memory offset and report a failure in the status
word instead of making the access.
"""
from __future__ import annotations

import glob
import os
import re
import shutil
import importlib.util
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libgqa_decode.so")
BUILD_CHECKED = os.path.join(ROOT, "_build_checked")
LIB_CHECKED = os.path.join(PKG, "libgqa_decode_checked.so")
CALLS = os.path.join(PKG, "_calls" + sysconfig.get_config_var("EXT_SUFFIX"))
CALLS_FOR = os.path.join(BUILD, "calls.for")     # what CALLS was built against
CALLS_SRC = os.path.join(CSRC, "torch_calls.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O3",
          "-I" + os.path.join(ROOT, "include"), "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (CUDA 13 toolkit required)")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))) + \
        [os.path.join(ROOT, "include", "gqa_decode.h"), os.path.abspath(__file__)]


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(p) <= t for p in _deps())


def _run(cmd, verbose: bool, what: str) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or r.returncode != 0:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed")


def torch_version() -> str:
    """Version of the installed torch, without importing it."""
    with open(os.path.join(os.path.dirname(importlib.util.find_spec("torch").origin), "version.py")) as f:
        return re.search(r"^__version__ = ['\"](.+?)['\"]", f.read(), re.M).group(1)


def _calls_for() -> str:
    return f"{importlib.util.find_spec('torch').origin} {torch_version()} {sys.version}"


def calls_up_to_date() -> bool:
    """The extension module is newer than its sources and was built against the torch that is installed."""
    if not os.path.exists(CALLS) or not os.path.exists(CALLS_FOR):
        return False
    with open(CALLS_FOR) as f:
        if f.read() != _calls_for():
            return False
    t = os.path.getmtime(CALLS)
    deps = [CALLS_SRC, os.path.join(ROOT, "include", "gqa_decode.h"), os.path.abspath(__file__),
            importlib.util.find_spec("torch").origin]
    return all(os.path.getmtime(p) <= t for p in deps)


def _compile_calls(verbose: bool) -> str:
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    obj = os.path.join(BUILD, "torch_calls.o")
    inc = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include"),
           sysconfig.get_paths()["include"], os.path.join(ROOT, "include")]
    _run(["g++", "-O2", "-std=c++17", "-fPIC", f'-DGQA_TORCH="{torch_version()}"'] + [f for p in inc for f in ("-isystem", p)] + ["-c", CALLS_SRC, "-o", obj],
         verbose, "g++ for torch_calls.cpp")
    return obj


def _link_calls(obj: str, verbose: bool) -> None:
    lib = os.path.join(os.path.dirname(importlib.util.find_spec("torch").origin), "lib")
    tmp = CALLS + ".tmp"
    _run(["g++", "-shared", "-o", tmp, obj, "-L" + lib, "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10_cuda", "-lc10",
          "-L" + PKG, "-lgqa_decode", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib], verbose,
         f"link of {os.path.basename(CALLS)}")
    os.replace(tmp, CALLS)
    with open(CALLS_FOR, "w") as f:
        f.write(_calls_for())


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False, checked: bool = False) -> str:
    """Compile and link the library (``checked``: the bounds-checked one); returns its path."""
    lib, bdir = (LIB_CHECKED, BUILD_CHECKED) if checked else (LIB, BUILD)
    os.makedirs(bdir, exist_ok=True)
    if checked:
        return _build_library(lib, bdir, force, verbose, ptxas_verbose, checked)
    with ThreadPoolExecutor(1) as ex:
        calls = ex.submit(_compile_calls, verbose) if force or not calls_up_to_date() else None
        _build_library(lib, bdir, force, verbose, ptxas_verbose, checked)
        if calls is not None:
            _link_calls(calls.result(), verbose)
    return lib


def _build_library(lib: str, bdir: str, force: bool, verbose: bool, ptxas_verbose: bool, checked: bool) -> str:
    if not force and up_to_date(lib):
        return lib
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_verbose else []
    if checked:
        extra += ["-DGQA_BOUNDS_CHECK=1"]

    def compile_one(src: str):
        obj = os.path.join(bdir, os.path.basename(src)[:-3] + ".o")
        cmd = [cc] + ARCH + CFLAGS + extra + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        return obj, cmd, r

    srcs = _sources()
    with ThreadPoolExecutor(max(1, min(len(srcs), os.cpu_count() or 1))) as ex:
        results = list(ex.map(compile_one, srcs))
    for obj, cmd, r in results:
        if verbose or ptxas_verbose or r.returncode != 0:
            sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {os.path.basename(obj)}")
    tmp = lib + ".tmp"
    cmd = [cc] + ARCH + ["-shared", "-o", tmp] + [o for o, _, _ in results] + ["-lpthread", "-ldl", "-lrt"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or r.returncode != 0:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError(f"link of {os.path.basename(lib)} failed")
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_verbose="-v" in sys.argv,
                checked="--checked" in sys.argv))
