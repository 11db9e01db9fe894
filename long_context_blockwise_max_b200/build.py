"""Build step of the native library: compiles csrc/*.cu for sm_100a into
``libpulsar_b200.so`` beside this file (in-tree, so it travels with the
source tree), and the serving operators' Python call layer (csrc/*.cpp, against
torch's headers) into ``call_layer_path()``.  Runs on a machine without a GPU:
nvcc cross-compiles.

    python -m long_context_blockwise_max_b200.build [--force] [--verbose]
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
LIB = os.path.join(PKG, "libpulsar_b200.so")
CALL_SRC = os.path.join(CSRC, "serving_call.cpp")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpulsar_b200.so")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
    deps += glob.glob(os.path.join(ROOT, "include", "*.h"))
    return any(os.path.getmtime(p) > t for p in deps)


def _compile(src: str, obj: str, ptxas_verbose: bool) -> subprocess.CompletedProcess:
    cmd = [_nvcc(), "-O3", "-std=c++17", *ARCH, "-lineinfo", "-Xcompiler", "-fPIC", "-c",
           "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include"), "-o", obj, src]
    if ptxas_verbose:
        cmd += ["-Xptxas", "-v"]
    return subprocess.run(cmd, capture_output=True, text=True)


def call_layer_path() -> str:
    """The call layer built for this Python and this torch: it uses both by
    their binary interfaces, which no other version need share."""
    import sysconfig

    import torch
    return os.path.join(PKG, f"_serving_call.torch-{torch.__version__}{sysconfig.get_config_var('EXT_SUFFIX')}")


def build_call_layer(force: bool = False) -> str:
    """Compile the Python call layer of the serving operators if there is none
    for this Python and torch, or a source or header of it is newer; return its
    path.  Links to the library built by ``build`` (found beside it at run time)."""
    call = call_layer_path()
    deps = [CALL_SRC] + glob.glob(os.path.join(ROOT, "include", "*.h"))
    if not force and os.path.exists(call) and all(os.path.getmtime(p) <= os.path.getmtime(call) for p in deps):
        return call
    import sysconfig

    import torch
    base = os.path.dirname(torch.__file__)
    inc = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")]
    lib = os.path.join(base, "lib")
    tmp = call + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-I{i}" for i in inc), CALL_SRC,
           "-o", tmp, f"-L{PKG}", "-l:" + os.path.basename(LIB), f"-L{lib}", "-ltorch_python", "-ltorch_cuda",
           "-ltorch_cpu", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("compiling the call layer failed")
    os.replace(tmp, call)
    return call


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    """Compile the library if a source is newer than it; return its path.
    Each .cu is compiled to an object in parallel under _build/, then linked."""
    if not force and not _stale():
        build_call_layer()
        return LIB
    from concurrent.futures import ThreadPoolExecutor
    bdir = os.path.join(ROOT, "_build")
    os.makedirs(bdir, exist_ok=True)
    srcs = sources()
    objs = [os.path.join(bdir, os.path.basename(s)[:-3] + ".o") for s in srcs]
    with ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 1))) as ex:
        results = list(ex.map(lambda so: _compile(so[0], so[1], ptxas_verbose), zip(srcs, objs)))
    failed = False
    for src, r in zip(srcs, results):
        if verbose or ptxas_verbose or r.returncode != 0:
            sys.stdout.write(r.stdout)
            sys.stderr.write(r.stderr)
        failed |= r.returncode != 0
    if failed:
        raise RuntimeError("nvcc failed")
    tmp = LIB + ".tmp"
    link = [_nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(link, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("nvcc link failed")
    os.replace(tmp, LIB)
    build_call_layer(force)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="--verbose" in sys.argv,
          ptxas_verbose="--ptxas" in sys.argv)
    print(LIB)
