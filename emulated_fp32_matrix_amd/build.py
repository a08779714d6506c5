"""Build the HIP library ``libemu_sgemm.so`` in-tree for gfx950, and the torch
binding of its block operators, ``_block_ops.so`` (host code).

Every ``csrc/*.hip`` file is compiled by hipcc to an object under
``_build/`` (in parallel, beside the binding's), then linked into the package
directory, where the Python binding loads it.  Always recompiles: this is the "does it build"
check as well as the build.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_NAME = "libemu_sgemm.so"
OPS_NAME = "_block_ops.so"
ARCH = "gfx950"

HIPCC_FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++20",
    "-fPIC",
    "-ffp-contract=off",            # every fused multiply-add is written out explicitly
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
]


def _hipcc() -> str:
    path = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(path):
        raise RuntimeError("hipcc not found (ROCm is required to build the library)")
    return path


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
    cmd = [_hipcc(), *HIPCC_FLAGS, "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-c", src,
           "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    err = "\n".join(line for line in r.stderr.splitlines()
                    if "packed-fp32-ops' is not a recognized feature" not in line)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{err}")
    if verbose and err.strip():
        print(err, flush=True)
    return obj


def _compile_ops(verbose: bool) -> str:
    """The torch binding's object: g++, torch's headers."""
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths

    src = os.path.join(CSRC, "block_torch.cpp")
    obj = os.path.join(BUILD_DIR, "block_torch.cpp.o")
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    dirs = [os.path.join(ROOT, "include"), *include_paths(), sysconfig.get_paths()["include"],
            os.path.join(rocm, "include")]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-Wall", "-Wno-attributes", "-Wno-unknown-pragmas",
           "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1", f"-DTORCH_EXTENSION_NAME={OPS_NAME.split('.')[0]}",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[f for d in dirs for f in ("-isystem" if d != dirs[0] else "-I", d)], "-c", src, "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {src}:\n{r.stderr}")
    if verbose and r.stderr.strip():
        print(r.stderr, flush=True)
    return obj


def _link_ops(obj: str, verbose: bool) -> None:
    import torch

    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    out = os.path.join(PKG, OPS_NAME)
    tmp = out + ".tmp"
    # libemu_sgemm.so lies beside it; torch's libraries are loaded before it
    cmd = ["g++", "-shared", "-fPIC", obj, "-o", tmp, os.path.join(PKG, LIB_NAME), "-Wl,-rpath,$ORIGIN", f"-L{libs}",
           "-lc10", "-lc10_hip", "-ltorch", "-ltorch_cpu", "-ltorch_python", os.path.join(libs, "libamdhip64.so")]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, out)


def build(verbose: bool = False) -> str:
    """Compile all sources and link the shared library and the torch binding;
    returns the library's path."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.hip")))
    with cf.ThreadPoolExecutor(max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        ops = ex.submit(_compile_ops, verbose)
        objs = list(ex.map(lambda s: _compile(s, verbose), srcs))
        ops_obj = ops.result()
    out = os.path.join(PKG, LIB_NAME)
    tmp = out + ".tmp"
    cmd = [_hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", f"-Wl,-soname,{LIB_NAME}", *objs, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, out)
    _link_ops(ops_obj, verbose)
    return out


if __name__ == "__main__":
    print(build(verbose=True))
