"""Build libgdr.so in-tree for sm_100a.

    python -m gated_deltanet_gdr_b200.build [--force] [--verbose-ptxas]

Each ``csrc/*.cu`` is compiled to an object with
``nvcc -gencode arch=compute_100a,code=sm_100a -O3 -lineinfo`` (in parallel) and
linked into ``gated_deltanet_gdr_b200/libgdr.so`` with the CUDA runtime linked
statically, so the library loads on a machine without a GPU driver (the driver is
only opened at the first CUDA call).  ``csrc/marshal.cpp``, the checks and marshalling
of the short calls for the Python binding, is compiled with g++ against the installed
torch, as an extension module of the running Python (``_marshal``); where that fails, a
warning says why, and the binding marshals those calls in Python.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import hashlib
import importlib.metadata
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libgdr.so")
MARSHAL = os.path.join(PKG, "_marshal" + sysconfig.get_config_var("EXT_SUFFIX"))
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-Xcompiler", "-Wall", "-diag-suppress", "177"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found; set NVCC or put the CUDA toolkit on PATH")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (_sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])


def up_to_date() -> bool:
    return _newer(LIB, _deps()) and _marshal_settled()


def _newer(target: str, deps) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(p) <= t for p in deps)


def _marshal_sources():
    return [os.path.join(CSRC, "marshal.cpp"), os.path.join(INCLUDE, "gdr.h"), os.path.abspath(__file__)]


def _marshal_key() -> str:
    """What the extension is made of: its sources and the torch whose headers it is compiled against."""
    h = hashlib.sha256()
    for p in _marshal_sources():
        with open(p, "rb") as f:
            h.update(f.read())
    try:
        torch_version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        torch_version = "none"
    return f"{h.hexdigest()} torch {torch_version}"


def _stamp() -> str:
    return os.path.join(OBJ, "marshal.stamp")


def _marshal_settled() -> bool:
    """Whether the extension of this key was built and is there, or could not be built."""
    try:
        with open(_stamp()) as f:
            key, outcome = f.read().rsplit(": ", 1)
    except (OSError, ValueError):
        return False
    return key == _marshal_key() and (outcome == "failed" or os.path.exists(MARSHAL))


def _build_marshal() -> None:
    """Builds the extension, which the binding can do without: a failure is reported, and not tried again before something
    changes (or with force)."""
    os.makedirs(OBJ, exist_ok=True)
    try:
        _compile_marshal()
        outcome = "built"
    except Exception as e:
        if os.path.exists(MARSHAL):
            os.remove(MARSHAL)  # it may not fit the library any more
        warnings.warn(f"the extension _marshal was not built (short calls are marshalled in Python; --force tries again): {e}")
        outcome = "failed"
    with open(_stamp(), "w") as f:
        f.write(f"{_marshal_key()}: {outcome}")


def _compile_marshal() -> None:
    import torch
    root = os.path.dirname(torch.__file__)
    tmp = MARSHAL + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DGDR_TORCH="{torch.__version__}"',
           "-I", sysconfig.get_paths()["include"],
           "-isystem", os.path.join(root, "include"), "-isystem", os.path.join(root, "include/torch/csrc/api/include"),
           os.path.join(CSRC, "marshal.cpp"), "-o", tmp, "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch",
           "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compiling marshal.cpp failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, MARSHAL)


def _compile(src: str, verbose_ptxas: bool) -> str:
    obj = os.path.join(OBJ, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, "-I", INCLUDE, "-c", src, "-o", obj]
    if verbose_ptxas:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    if verbose_ptxas:
        sys.stderr.write(r.stderr)
    return obj


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    if not force and _newer(LIB, _deps()):
        _build_marshal()
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        marshal = None if not force and _marshal_settled() else ex.submit(_build_marshal)
        objs = list(ex.map(lambda s: _compile(s, verbose_ptxas), srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", *objs, "-o", tmp, "-ldl", "-lpthread", "-lrt"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if marshal is not None:
        marshal.result()
    return LIB


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose-ptxas", action="store_true", help="print registers/spills per kernel")
    args = ap.parse_args(argv)
    print(build(force=args.force, verbose_ptxas=args.verbose_ptxas))


if __name__ == "__main__":
    main()
