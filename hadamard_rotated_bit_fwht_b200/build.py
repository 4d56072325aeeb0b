"""Build the sm_100a shared library libkvq.so in-tree with nvcc.

    python -m hadamard_rotated_bit_fwht_b200.build
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libkvq.so")
# the same sources compiled with KVQ_DEBUG_BOUNDS: every computed cache,
# slot and scale-row address is checked against its buffer, and a violation
# is recorded in the device error word (kvq_device_errors) instead of accessed
LIB_DEBUG = os.path.join(PKG, "libkvq_debug.so")

# the binding's marshalling module (host code, built against torch)
BIND = os.path.join(PKG, "kvq_bind.so")

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "--shared", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-Xptxas", "-warn-spills",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + [os.path.join(INCLUDE, "kvq.h")]
    return any(os.path.getmtime(p) > t for p in deps)


OBJ_DIR = os.path.join(ROOT, "_build", "kvq")


def _cuda_include() -> str:
    """The headers beside nvcc, which may be a name on the PATH or a link."""
    nvcc = shutil.which(NVCC) or NVCC
    for p in (nvcc, os.path.realpath(nvcc)):
        inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(p))), "include")
        if os.path.exists(os.path.join(inc, "cuda_runtime_api.h")):
            return inc
    raise FileNotFoundError(f"no cuda_runtime_api.h in the include folder of {nvcc}")


def bind_key() -> str:
    """The Python and torch that a marshalling module belongs to."""
    import sysconfig

    import torch
    return (f"kvq_bind for {sysconfig.get_config_var('SOABI')}, torch {torch.__version__} "
            f"abi {int(torch.compiled_with_cxx11_abi())}")


def bind_is_for(key: str) -> bool:
    """Whether kvq_bind.so is there and was built for `key`, which it holds."""
    if not os.path.exists(BIND):
        return False
    with open(BIND, "rb") as f:
        return key.encode() + b"\0" in f.read()


def build_bind(force: bool = False) -> str:
    """Compile the marshalling module kvq_bind.so against the running Python and
    torch (host code only)."""
    import sysconfig

    import torch
    src = os.path.join(CSRC, "kvq_bind.cpp")
    if not force and bind_is_for(bind_key()) and all(
            os.path.getmtime(p) <= os.path.getmtime(BIND)
            for p in (src, os.path.join(INCLUDE, "kvq.h"))):
        return BIND
    t = os.path.dirname(torch.__file__)
    inc = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(t, "include"),
           os.path.join(t, "include", "torch", "csrc", "api", "include"),
           _cuda_include()]
    tmp = BIND + f".tmp{os.getpid()}"
    subprocess.check_call([
        "g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", "-w",
        f'-DKVQ_BIND_KEY="{bind_key()}"',
        f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
        *(f"-I{p}" for p in inc), src, "-o", tmp, "-L" + os.path.join(t, "lib"),
        "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"])
    os.replace(tmp, BIND)
    return BIND


def build(force: bool = False, verbose: bool = False, debug: bool = False) -> str:
    """Compile every .cu to an object in parallel (relocatable device code is
    not needed: no kernel calls across files), then link libkvq.so (or, with
    debug=True, libkvq_debug.so with the bounds checks compiled in).  Then, where
    there is a torch to build it against, the marshalling module of the Python
    binding: the library itself needs nvcc alone."""
    lib = LIB_DEBUG if debug else LIB
    if force or _stale(lib):
        _build_lib(lib, verbose, debug)
    try:
        import torch  # noqa: F401
    except ImportError:
        print("no torch: the module of the Python binding is not built", file=sys.stderr)
    else:
        build_bind(force and not debug)
    return lib


def _build_lib(lib: str, verbose: bool, debug: bool) -> None:
    from concurrent.futures import ThreadPoolExecutor
    os.makedirs(OBJ_DIR, exist_ok=True)
    compile_flags = [f for f in FLAGS if f not in ("--shared",)]
    if debug:
        compile_flags += ["-DKVQ_DEBUG_BOUNDS"]
    tag = f".{'dbg' if debug else 'rel'}{os.getpid()}"

    def compile_one(src):
        obj = os.path.join(OBJ_DIR, os.path.basename(src)[:-3] + tag + ".o")
        cmd = [NVCC, *compile_flags, "-I", INCLUDE, "-c", src, "-o", obj]
        if verbose:
            cmd += ["-Xptxas", "-v"]
            print(" ".join(cmd))
        subprocess.check_call(cmd)
        return obj

    srcs = sources()
    with ThreadPoolExecutor(min(len(srcs), os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = lib + f".tmp{os.getpid()}"
    subprocess.check_call([NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "--shared",
                           "-Xcompiler", "-fPIC", "-o", tmp, *objs])
    os.replace(tmp, lib)
    for o in objs:
        os.remove(o)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                debug="--debug" in sys.argv))
