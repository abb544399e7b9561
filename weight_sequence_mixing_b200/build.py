"""Build step of the CUDA library: compiles csrc/*.cu for sm_100a with nvcc and
links them, with the static CUDA runtime, into libttt_b200.so next to this file; then
the Python module _token_ops (csrc/token_ops_py.cpp), which calls it on torch tensors.

Object files go to ../_build (ignored by git); a source whose text and flags are
unchanged since the last build is not recompiled.
"""
from __future__ import annotations

import glob
import hashlib
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libttt_b200.so")
MODULE = os.path.join(PKG, "_token_ops.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ARCH + ["-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "--expt-relaxed-constexpr",
                     "-I", INCLUDE, "-I", CSRC]


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA library cannot be built")


def _digest(path: str, flags: list[str]) -> str:
    h = hashlib.sha256()
    h.update(" ".join(flags).encode())
    headers = [g for d, e in ((CSRC, "*.cuh"), (CSRC, "*.h"), (INCLUDE, "*.h")) for g in glob.glob(os.path.join(d, e))]
    for f in sorted(headers + [path]):
        h.update(f.encode())
        with open(f, "rb") as fh:
            h.update(fh.read())
    return h.hexdigest()[:16]


def build(verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    """Compile every csrc/*.cu and link libttt_b200.so; returns the library path."""
    nvcc = nvcc_path()
    flags = NVCC_FLAGS + list(extra_flags or [])
    os.makedirs(BUILD, exist_ok=True)
    objs, todo = [], []
    for src in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        name = os.path.splitext(os.path.basename(src))[0]
        obj = os.path.join(BUILD, f"{name}.{_digest(src, flags)}.o")
        if not os.path.exists(obj):
            todo.append([nvcc] + flags + ["-c", src, "-o", obj])
        objs.append(obj)
    changed = bool(todo)

    def compile_one(cmd):
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        try:
            subprocess.run(cmd, check=True)
        except BaseException:
            if os.path.exists(cmd[-1]):
                os.remove(cmd[-1])  # a part of an object is not one
            raise

    with ThreadPoolExecutor(max_workers=os.cpu_count() or 1) as pool:
        list(pool.map(compile_one, todo))
    # the objects the library was last linked from: relink whenever they differ (a
    # source reverted to an earlier version finds its old object in the cache)
    manifest = os.path.join(BUILD, "libttt_b200.objects")
    listing = "\n".join(os.path.basename(o) for o in objs)
    linked = open(manifest).read() if os.path.exists(manifest) else None
    if changed or linked != listing or not os.path.exists(LIB):
        tmp = LIB + ".tmp"
        cmd = [nvcc] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        subprocess.run(cmd, check=True)
        os.replace(tmp, LIB)
        with open(manifest, "w") as f:
            f.write(listing)
    return LIB


def build_module(verbose: bool = False) -> str:
    """Compile and link the Python module _token_ops against torch and libttt_b200.so; returns its path."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    src = os.path.join(CSRC, "token_ops_py.cpp")
    cuda = os.path.dirname(os.path.dirname(nvcc_path()))
    includes = [sysconfig.get_paths()["include"], INCLUDE, os.path.join(cuda, "include")] + cpp_extension.include_paths()
    flags = ["-std=c++17", "-O2", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    flags += [f for d in includes for f in ("-isystem", d)]
    flags += [f"-L{d}" for d in cpp_extension.library_paths()]
    libs = ["-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10", f"-L{PKG}", "-l:libttt_b200.so",
            "-Wl,-rpath,$ORIGIN"]
    built = os.path.join(BUILD, f"_token_ops.{_digest(src, flags + libs + [torch.__version__, sys.version])}.so")
    if not os.path.exists(built):
        cmd = ["g++"] + flags + ["-o", built + ".tmp", src] + libs
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        subprocess.run(cmd, check=True)
        os.replace(built + ".tmp", built)
    if not os.path.exists(MODULE) or open(MODULE, "rb").read() != open(built, "rb").read():
        shutil.copyfile(built, MODULE + ".tmp")
        os.replace(MODULE + ".tmp", MODULE)
    return MODULE


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
    print(build_module(verbose="-v" in sys.argv))
