"""Build libkvc.so in place with nvcc for sm_100a (no JIT cache: the library sits
beside this file so it travels with the source tree)."""
from __future__ import annotations

import glob
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libkvc.so")
BIND = os.path.join(HERE, "_bind.so")  # csrc/bind.cpp, loaded by kvc.py
BIND_FOR = os.path.join(HERE, "_build", "bind_for.txt")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr"]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _bind_target() -> str:
    """The torch and interpreter that _bind.so is compiled for (kept beside its build in BIND_FOR)."""
    import torch

    return f"torch {torch.__version__}, {sys.implementation.cache_tag}"


def _newer(target: str, deps) -> bool:
    deps = list(deps) + [os.path.join(HERE, "..", "include", "kvc.h")]
    return os.path.exists(target) and all(os.path.getmtime(d) <= os.path.getmtime(target) for d in deps if os.path.exists(d))


def lib_up_to_date() -> bool:
    return _newer(LIB, sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")))


def bind_up_to_date() -> bool:
    if not _newer(BIND, [os.path.join(CSRC, "bind.cpp")]) or not os.path.exists(BIND_FOR):
        return False
    with open(BIND_FOR) as f:
        return f.read() == _bind_target()


def up_to_date() -> bool:
    return lib_up_to_date() and bind_up_to_date()


def build(force: bool = False, verbose: bool = False, jobs: int = 8) -> str:
    """Compile every csrc/*.cu for sm_100a and link libkvc.so, and compile _bind.so; returns the library's path.  The library is all
    that is needed: where _bind.so does not compile (no headers of torch or Python), that is said and the Python path is left."""
    if not force and up_to_date():
        return LIB
    os.makedirs(os.path.join(HERE, "_build"), exist_ok=True)
    bind = None if not force and bind_up_to_date() else _start_bind(BIND + ".tmp")
    if force or not lib_up_to_date():
        _build_lib(verbose, jobs)
    if bind is not None:
        _finish_bind(bind)
    return LIB


def _build_lib(verbose: bool, jobs: int):
    procs, objs = [], []
    for src in sources():
        obj = os.path.join(HERE, "_build", os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        cmd = [NVCC, *ARCH, *FLAGS, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
        if len(procs) >= jobs:
            _reap(procs, verbose)
    _reap(procs, verbose)
    tmp = LIB + ".tmp"
    link = [NVCC, *ARCH, "-shared", "-o", tmp, *objs]
    out = subprocess.run(link, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if out.returncode != 0:
        raise RuntimeError("link failed:\n" + out.stdout)
    os.replace(tmp, LIB)


def _start_bind(out: str):
    """Start compiling csrc/bind.cpp against torch's headers and libraries (those of the interpreter that builds)."""
    import sysconfig

    import torch

    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(NVCC))
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DKVC_TORCH="{torch.__version__}"',
           f"-I{root}/include", f"-I{root}/include/torch/csrc/api/include", f"-I{cuda}/include",
           f"-I{sysconfig.get_paths()['include']}", "-o", out, os.path.join(CSRC, "bind.cpp"), f"-L{root}/lib",
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", f"-Wl,-rpath,{root}/lib"]
    try:
        return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    except OSError as e:
        return e


def _finish_bind(proc):
    """Put _bind.so in its place, or, if it did not compile, say so and leave none (an older one may not fit the library)."""
    out = str(proc) if isinstance(proc, OSError) else proc.communicate()[0]
    if not isinstance(proc, OSError) and proc.returncode == 0:
        os.replace(BIND + ".tmp", BIND)
        with open(BIND_FOR, "w") as f:
            f.write(_bind_target())
        return
    for path in (BIND, BIND_FOR):
        if os.path.exists(path):
            os.remove(path)
    sys.stderr.write("_bind.so was not built (calls are packed in Python instead):\n" + out + "\n")


def _reap(procs, verbose):
    errs = []
    for src, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            errs.append(f"{src}:\n{out}")
        elif verbose and out:
            sys.stderr.write(out)
    procs.clear()
    if errs:
        raise RuntimeError("nvcc failed:\n" + "\n".join(errs))


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
