"""Build libqlin.so in-tree with nvcc for sm_103a (GB300).

Each .cu file under csrc/ is compiled to an object in parallel, then linked
into ``w4a16_linear_layers_gb300/_build/libqlin.so``.  The library links the
CUDA runtime statically and reaches the driver's tensor-map encoder through
the runtime's entry-point query, so it does not link against PyTorch or
libcuda.  csrc/torch_calls.cpp, the Python extension of the calls that are
short on the device, becomes ``_build/qlin_torch.so`` beside it, with the host
compiler and PyTorch's headers, and ``qlin_torch.stamp`` says which PyTorch and
Python it is for.  The library does not wait for it: it is there without
PyTorch, and where the extension cannot be built.  Usage:
``python -m w4a16_linear_layers_gb300.build [--force]``.
"""
from __future__ import annotations

import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(BUILD_DIR, "libqlin.so")
CALLS_PATH = os.path.join(BUILD_DIR, "qlin_torch.so")
CALLS_SOURCE = os.path.join(CSRC, "torch_calls.cpp")
INCLUDE = os.path.join(ROOT, "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _newer(path: str, deps) -> bool:
    """path is there and none of deps changed after it."""
    return os.path.exists(path) and all(os.path.getmtime(d) <= os.path.getmtime(path) for d in deps)


def _library_up_to_date() -> bool:
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    deps = [d for d in deps if d != CALLS_SOURCE]
    return _newer(LIB_PATH, deps + [os.path.join(INCLUDE, "qlin.h"), os.path.abspath(__file__)])


def calls_stamp() -> str | None:
    """What the extension is built for; None where there is no PyTorch."""
    if importlib.util.find_spec("torch") is None:
        return None
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:     # in the path, not installed
        import torch

        version = torch.__version__
    return f"torch {version}, python {sysconfig.get_config_var('SOABI')}"


def calls_built_for() -> str | None:
    try:
        with open(os.path.splitext(CALLS_PATH)[0] + ".stamp") as f:
            return f.read()
    except OSError:
        return None


def _calls_up_to_date() -> bool:
    return (calls_built_for() == calls_stamp()
            and _newer(CALLS_PATH, [CALLS_SOURCE, os.path.join(INCLUDE, "qlin.h"), os.path.abspath(__file__)]))


def up_to_date() -> bool:
    return _library_up_to_date() and (calls_stamp() is None or _calls_up_to_date())


def _build_calls() -> None:
    base = os.path.dirname(importlib.util.find_spec("torch").origin)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    headers = [sysconfig.get_paths()["include"], os.path.join(base, "include"),
               os.path.join(base, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include")]
    tmp = CALLS_PATH + f".{os.getpid()}.tmp"
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-fvisibility=hidden", "-I", INCLUDE]
    for path in headers:
        cmd += ["-isystem", path]
    cmd += [CALLS_SOURCE, "-o", tmp, "-L", os.path.join(base, "lib"),
            "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for torch_calls.cpp:\n{r.stdout}\n{r.stderr}")
    stamp = os.path.splitext(CALLS_PATH)[0] + ".stamp"
    if os.path.exists(stamp):      # none while the extension changes
        os.remove(stamp)
    os.replace(tmp, CALLS_PATH)
    with open(stamp + f".{os.getpid()}.tmp", "w") as f:
        f.write(calls_stamp())
    os.replace(stamp + f".{os.getpid()}.tmp", stamp)


def _build_library(verbose: bool, extra_flags) -> None:
    cc = nvcc()
    flags = NVCC_FLAGS + list(extra_flags or [])
    srcs = _sources()

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *ARCH, *flags, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)
        return obj

    with ThreadPoolExecutor(max(1, min(len(srcs), os.cpu_count() or 1))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB_PATH + f".{os.getpid()}.tmp"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)


def build(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    """The library, then what is left of the extension: an error of the latter
    is raised when the former is in place."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    with ThreadPoolExecutor(1) as ex:      # beside the library
        calls = (ex.submit(_build_calls) if calls_stamp() is not None and (force or not _calls_up_to_date())
                 else None)
        if force or not _library_up_to_date():
            _build_library(verbose, extra_flags)
    if calls is not None and calls.exception() is not None:
        raise RuntimeError(f"{LIB_PATH} is built, its Python extension is not") from calls.exception()
    return LIB_PATH


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv,
          extra_flags=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else None)
    print(LIB_PATH)
