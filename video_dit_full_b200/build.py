"""Build the C-ABI library ``libwan_attn.so`` in-tree with nvcc for sm_100a.

    python -m video_dit_full_b200.build [--verbose]

Extra nvcc flags (tuning macros such as -DWAN_FWD_POLY_PAIRS=3) can be passed
in the WAN_ATTN_NVCC_FLAGS environment variable; use --force after changing it.
Each ``csrc/*.cu`` is compiled to an object under ``_build/`` (skipped when
up to date) and the objects are linked into ``video_dit_full_b200/libwan_attn.so``.
``csrc/bind.cpp``, the Python binding of the calls whose arguments are looked at
in C++, is compiled with g++ against PyTorch into ``video_dit_full_b200/_bind.*.so``,
named after the interpreter and the PyTorch that it is built for.
"""
from __future__ import annotations

import argparse
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "libwan_attn.so")
BUILD_DIR = os.path.join(ROOT, "_build")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def build_binding(force: bool = False) -> str | None:
    """The CPython extension ``_bind`` (no device code; the CUDA library is not linked in).  Without PyTorch
    there is nothing to bind for: None, and the C ABI is complete all the same."""
    try:
        import torch
    except ImportError:
        print("no PyTorch: the Python binding is not built", file=sys.stderr)
        return None

    from .wan_attn import binding_path
    out = binding_path()
    src, header = os.path.join(CSRC, "bind.cpp"), os.path.join(ROOT, "include", "wan_attn.h")
    if not force and os.path.exists(out) and os.path.getmtime(out) >= max(os.path.getmtime(src), os.path.getmtime(header)):
        return out
    at = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    tmp = out + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", os.path.join(ROOT, "include")]
    for d in (at, os.path.join(at, "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"], cuda):
        cmd += ["-isystem", d]
    cmd += [src, "-o", tmp, "-L", os.path.join(os.path.dirname(at), "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
            "-ltorch_cuda", "-ltorch_python"]
    print(" ".join(cmd), file=sys.stderr)
    subprocess.check_call(cmd)
    os.replace(tmp, out)
    return out


def build(verbose: bool = False, force: bool = False) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    headers = glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))
    newest_header = max((os.path.getmtime(h) for h in headers), default=0)
    objs = []
    for src in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if (not force and os.path.exists(obj) and os.path.getmtime(obj) >= os.path.getmtime(src)
                and os.path.getmtime(obj) >= newest_header):
            continue
        cmd = [nvcc(), *ARCH, *FLAGS, *os.environ.get("WAN_ATTN_NVCC_FLAGS", "").split(), "-c", src, "-o", obj]
        if verbose:
            cmd += ["-Xptxas", "-v"]
        print(" ".join(cmd), file=sys.stderr)
        subprocess.check_call(cmd)
    if force or not os.path.exists(OUT) or any(os.path.getmtime(o) > os.path.getmtime(OUT) for o in objs):
        tmp = OUT + f".tmp{os.getpid()}"
        subprocess.check_call([nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-lcudart_static"])
        os.replace(tmp, OUT)
    build_binding(force)
    return OUT


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--force", action="store_true")
    a = ap.parse_args()
    print(build(verbose=a.verbose, force=a.force))
