"""Compile the CUDA sources of this package into libsparse_attn.so (in-tree), and
the CPython module that kv8.py calls it through.

nvcc cross-compiles for sm_100a without a GPU; the shared libraries land next
to this file, where the bindings load them.
"""

from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libsparse_attn.so")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "--expt-relaxed-constexpr", "-Xptxas", "-warn-spills"]


EXT_SRC = os.path.join(CSRC, "ext", "kv8_ext.cpp")
EXT = os.path.join(HERE, "_kv8_ext.so")


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found")
    return path


def sources() -> list:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _stale(obj: str, src: str) -> bool:
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    deps = [src] + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    deps.append(os.path.join(HERE, "..", "include", "sparse_attn.h"))
    return any(os.path.getmtime(d) > t for d in deps if os.path.exists(d))


def build(verbose: bool = False, force: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    objs, jobs = [], []
    for src in sources():
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, src):
            jobs.append([nvcc(), *ARCH, *FLAGS, "-c", src, "-o", obj])

    torch = _torch()
    ext_obj, ext_for = os.path.join(BUILD, "kv8_ext.o"), os.path.join(BUILD, "kv8_ext.torch")
    ext_stale = torch and (force or _stale(ext_obj, EXT_SRC) or _text(ext_for) != torch.__version__)
    with concurrent.futures.ThreadPoolExecutor(max_workers=max(1, len(jobs) + 1)) as ex:
        ext = ex.submit(_run, _ext_compile(torch, ext_obj)) if ext_stale else None
        for out in ex.map(_run, jobs):
            if verbose and out.strip():
                print(out)
        if jobs or not os.path.exists(LIB):
            _run([nvcc(), *ARCH, "-shared", "-o", LIB, *objs, "-lcudart"])
        if ext:
            ext.result()
    if torch and (ext_stale or not os.path.exists(EXT)):
        _run(_ext_link(torch, ext_obj))
        with open(ext_for, "w") as f:
            f.write(torch.__version__)
    if verbose and not torch:
        print("no torch with CUDA here: _kv8_ext.so is not built")
    return LIB


def _torch():
    """The torch that the CPython module is built against, or None: the C library needs none."""
    try:
        import torch
    except ImportError:
        return None
    return torch if torch.version.cuda else None


def _text(path: str) -> str:
    if not os.path.exists(path):
        return ""
    with open(path) as f:
        return f.read()


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
    return r.stdout + r.stderr


def _ext_compile(torch, obj: str) -> list:
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    return ["g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", cuda,
            "-isystem", sysconfig.get_paths()["include"], "-c", EXT_SRC, "-o", obj]


def _ext_link(torch, obj: str) -> list:
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    return ["g++", "-shared", "-o", EXT, obj, "-L" + HERE, "-l:libsparse_attn.so", "-L" + lib, "-ltorch_python",
            "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib]


if __name__ == "__main__":
    print(build(verbose=True, force="--force" in sys.argv))
