"""Build the sm_100a shared library in-tree: paged_head_latent_mla_b200/libmla_b200.so.

Run as ``python -m paged_head_latent_mla_b200._build``.  nvcc cross-compiles for
sm_100a without a GPU present.  The library needs nvcc alone; the Python binding's native
part is built after it where torch is installed (``--library-only``: not at all).
"""

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libmla_b200.so")
SOURCES = ["api.cu", "mla_attn.cu", "state_ops.cu", "spec_ops.cu", "plan.cpp", "noalloc.cu"]
MARSHAL_SOURCE = os.path.join(CSRC, "marshal.cpp")  # the Python binding's argument checks
HEADERS = ["mla_internal.h", "mla_launch.h", "sm100_ptx.cuh"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _older(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def needs_build() -> bool:
    return _older(LIB, [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [os.path.join(ROOT, "include", "mla.h")])


def marshal_path() -> str:
    """The binding's native part for this Python and torch.  It reads both's objects by their
    layout, so another version's file must neither count as built nor be loaded: the name
    says which ones it is for."""
    import torch

    return os.path.join(PKG, "_marshal.torch-%s.%s.so" % (torch.__version__, sysconfig.get_config_var("SOABI")))


def build_marshal(force: bool = False) -> str:
    """Compile the binding's native part against the installed torch (host code only)."""
    import torch

    target = marshal_path()
    if not force and not _older(target, [MARSHAL_SOURCE, os.path.join(ROOT, "include", "mla.h")]):
        return target
    home = os.path.dirname(torch.__file__)
    inc = [os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(nvcc_path())), "include")]
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch.compiled_with_cxx11_abi())]
    for d in inc:
        cmd += ["-isystem", d]
    cmd += [MARSHAL_SOURCE, "-o", target + ".tmp"]
    cmd += ["-L" + os.path.join(home, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("g++ failed:\n" + res.stdout + res.stderr)
    os.replace(target + ".tmp", target)
    return target


def build(force: bool = False, verbose: bool = False, library_only: bool = False) -> str:
    """Build what is missing or older than its sources: the library, then the binding's native
    part unless ``library_only`` (or without torch, which the binding cannot do without)."""
    if force or needs_build():
        _build_library(verbose)
    if not library_only:
        if importlib.util.find_spec("torch") is None:
            sys.stderr.write("torch is not installed: only the library was built, not the Python binding's part\n")
        else:
            build_marshal(force)
    return LIB


def _build_library(verbose: bool) -> None:
    cmd = [
        nvcc_path(),
        "-gencode", "arch=compute_100a,code=sm_100a",
        "-lineinfo", "-O3", "-std=c++17",
        "-shared", "-Xcompiler", "-fPIC,-O2",
        "-I", os.path.join(ROOT, "include"),
        "-o", LIB + ".tmp",
    ] + [os.path.join(CSRC, f) for f in SOURCES]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + res.stdout + res.stderr)
    if verbose:
        sys.stderr.write(res.stderr)
    os.replace(LIB + ".tmp", LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, library_only="--library-only" in sys.argv))
