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


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(BIND) or not os.path.exists(BIND_FOR):
        return False
    with open(BIND_FOR) as f:
        if f.read() != _bind_target():
            return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(BIND))
    deps = sources() + [os.path.join(CSRC, "bind.cpp")] + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
    deps.append(os.path.join(HERE, "..", "include", "kvc.h"))
    return all(os.path.getmtime(d) <= t for d in deps if os.path.exists(d))


def build(force: bool = False, verbose: bool = False, jobs: int = 8) -> str:
    """Compile every csrc/*.cu for sm_100a and link libkvc.so, and compile _bind.so; returns the library's path."""
    if not force and up_to_date():
        return LIB
    objdir = os.path.join(HERE, "_build")
    os.makedirs(objdir, exist_ok=True)
    procs, objs = [], []
    procs.append(("bind.cpp", _start_bind(BIND + ".tmp")))
    for src in sources():
        obj = os.path.join(objdir, os.path.basename(src)[:-3] + ".o")
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
    os.replace(BIND + ".tmp", BIND)
    with open(BIND_FOR, "w") as f:
        f.write(_bind_target())
    return LIB


def _start_bind(out: str):
    """Compile csrc/bind.cpp against torch's headers and libraries (those of the interpreter that builds)."""
    import sysconfig

    import torch

    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(NVCC))
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DKVC_TORCH="{torch.__version__}"',
           f"-I{root}/include", f"-I{root}/include/torch/csrc/api/include", f"-I{cuda}/include",
           f"-I{sysconfig.get_paths()['include']}", "-o", out, os.path.join(CSRC, "bind.cpp"), f"-L{root}/lib",
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", f"-Wl,-rpath,{root}/lib"]
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)


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
