"""Builds libkda.so in-tree from csrc/*.cu for sm_103a with nvcc, and the binding's
checks of arguments, _host_args.so (with Python's tag in its name), from
csrc/host_args.cpp with g++ and PyTorch's headers.

Each translation unit is compiled in parallel, then linked into one shared
library next to this file.  Rebuilds only when a source is newer than the
library, or when the binding's checks were built for another PyTorch or Python:
they read tensors by PyTorch's own layout.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sysconfig
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libkda.so")
HOST = os.path.join(HERE, "_host_args" + sysconfig.get_config_var("EXT_SUFFIX"))
HOST_FOR = os.path.join(HERE, "_host_args.built_for")  # made_for() of its build
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    deps = srcs + sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")))
    deps += [os.path.join(os.path.dirname(HERE), "include", "kda.h"), os.path.join(CSRC, "host_args.cpp")]
    return srcs, deps


def _host_command(out):
    import torch

    root = os.path.dirname(torch.__file__)
    include, lib = os.path.join(root, "include"), os.path.join(root, "lib")
    headers = (sysconfig.get_paths()["include"], include, os.path.join(include, "torch", "csrc", "api", "include"))
    return [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-Wall", "-Wextra",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(x for h in headers for x in ("-isystem", h)),
            os.path.join(CSRC, "host_args.cpp"), "-o", out, "-L", lib, "-ltorch_python", "-ltorch_cpu", "-lc10"]


def made_for() -> str:
    """What the binding's checks are built against."""
    import torch

    return f"PyTorch {torch.__version__}, C++ ABI {int(torch._C._GLIBCXX_USE_CXX11_ABI)}, {os.path.basename(HOST)}"


def built_for() -> str | None:
    """made_for() of the build that is there, if one is."""
    try:
        with open(HOST_FOR) as f:
            return f.read()
    except OSError:
        return None


def stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(HOST) or built_for() != made_for():
        return True
    _, deps = _sources()
    t = min(os.path.getmtime(LIB), os.path.getmtime(HOST))
    return any(os.path.getmtime(d) > t for d in deps if os.path.exists(d))


def install(src: str, dst: str) -> None:
    """src as dst, by a copy beside dst and a rename: a process that has the old file
    mapped keeps it whole."""
    tmp = f"{dst}.{os.getpid()}"
    try:
        shutil.copy(src, tmp)
        os.replace(tmp, dst)
    finally:
        if os.path.exists(tmp):
            os.remove(tmp)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not stale():
        return LIB
    nvcc = _nvcc()
    srcs, _ = _sources()
    with tempfile.TemporaryDirectory(prefix="kda_build_") as tmp:
        procs, objs = [], []
        for s in srcs:
            obj = os.path.join(tmp, os.path.basename(s)[:-3] + ".o")
            objs.append(obj)
            cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-c", s, "-o", obj]
            if verbose:
                print(" ".join(cmd))
            procs.append((cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
        host = os.path.join(tmp, "_host_args.so")
        cmd = _host_command(host)
        procs.append((cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
        failed = []
        for cmd, p in procs:
            out, _ = p.communicate()
            if p.returncode != 0:
                failed.append((cmd, out.decode(errors="replace")))
        if failed:
            raise RuntimeError("compilation failed:\n" + "\n".join(" ".join(c) + "\n" + o for c, o in failed))
        tmp_lib = os.path.join(tmp, "libkda.so")
        subprocess.check_call([nvcc, *ARCH, "-shared", "-o", tmp_lib, *objs])
        for old in (HOST_FOR, os.path.join(HERE, "_host_args.so")):  # (any Python would import one without a tag)
            if os.path.exists(old):
                os.remove(old)
        install(host, HOST)
        with open(HOST_FOR, "w") as f:
            f.write(made_for())
        install(tmp_lib, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
