"""Build libmoe.so (the CUDA library behind include/moe_cache.h) in-tree for sm_100a, and the
extension module that marshals torch tensors for its attention operators."""
from __future__ import annotations

import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT_DIR = os.path.join(PKG, "_lib")
LIB = os.path.join(OUT_DIR, "libmoe.so")
BIND = os.path.join(OUT_DIR, "_moe_bind.so")
BIND_SRC = os.path.join(CSRC, "bind.cpp")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden",
         "--expt-relaxed-constexpr", f"-I{os.path.join(ROOT, 'include')}"]


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(ROOT, "include", "*.h"))
    return any(os.path.getmtime(d) > t for d in deps)


def _build_bind(force: bool) -> None:
    """The extension module, where torch and its headers are there (the library needs neither).  Rebuilt
    when its sources, torch or the interpreter are other ones."""
    import sysconfig
    try:
        import torch
        from torch.utils.cpp_extension import include_paths, library_paths
    except ImportError:
        return
    if not any(os.path.exists(os.path.join(i, "torch", "extension.h")) for i in include_paths()):
        return
    deps = [BIND_SRC, os.path.join(ROOT, "include", "moe_cache.h")]
    made_with = f"{torch.__version__} {sysconfig.get_config_var('SOABI')}\n"
    stamp = BIND + ".stamp"
    if not force and os.path.exists(BIND) and os.path.getmtime(BIND) >= max(os.path.getmtime(d) for d in deps):
        if os.path.exists(stamp):
            with open(stamp) as f:
                if f.read() == made_with:
                    return
    inc = include_paths() + [sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include"),
                             os.path.join(ROOT, "include")]
    tmp = BIND + f".{os.getpid()}.tmp"
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-DTORCH_EXTENSION_NAME=_moe_bind",
                           "-DTORCH_API_INCLUDE_EXTENSION_H", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
                           *[f"-I{i}" for i in inc], BIND_SRC, "-o", tmp, *[f"-L{p}" for p in library_paths()], f"-L{OUT_DIR}",
                           "-l:libmoe.so", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python", "-Wl,-rpath,$ORIGIN"])
    os.replace(tmp, BIND)
    with open(stamp + f".{os.getpid()}.tmp", "w") as f:
        f.write(made_with)
    os.replace(f.name, stamp)


def build(force: bool = False, verbose: bool = False) -> str:
    if force or _stale():
        _build_lib(verbose)
    _build_bind(force)
    return LIB


def _build_lib(verbose: bool) -> None:
    os.makedirs(OUT_DIR, exist_ok=True)
    objs = []
    for src in sources():
        obj = os.path.join(OUT_DIR, os.path.basename(src) + ".o")
        cmd = [NVCC, *ARCH, *FLAGS, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        subprocess.check_call(cmd)
        objs.append(obj)
    tmp = LIB + f".{os.getpid()}.tmp"
    subprocess.check_call([NVCC, *ARCH, "-shared", "-o", tmp, *objs, "-lpthread", "-ldl", "-lrt"])
    os.replace(tmp, LIB)
    for o in objs:
        os.remove(o)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
