"""Build libdtcoll.so (the HIP library behind include/dt.h) in-tree for gfx950.

    python collective_communication_primitives_amd/build.py

(Run by path: importing the package loads the library, which may be the
stale build this script replaces.)

Each source is compiled on its own (in parallel) into ``_build/`` at the
repository root, then linked into ``libdtcoll.so`` next to this file.  Beside
it ``_marshal`` with the suffix of this Python's extensions, the host helper of
the model-step operators' binding (g++, no GPU code).
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIBRARY = os.path.join(PKG, "libdtcoll.so")
MARSHAL = os.path.join(PKG, "_marshal" + sysconfig.get_config_var("EXT_SUFFIX"))
SOURCES = ("api.cpp", "reduce.hip", "copy.hip", "barrier.hip", "scratch.hip", "step_api.cpp", "norm.hip", "moe.hip",
           "loss.hip")
ARCH = os.environ.get("DT_OFFLOAD_ARCH", "gfx950")

HIPCC_FLAGS = [
    "-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
    # packed fp32 instructions stay off: plain float code only
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-result",
    "-I", INCLUDE, "-I", CSRC,
]


def _hipcc() -> str:
    return shutil.which("hipcc") or "/opt/rocm/bin/hipcc"


def _compile(src: str) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [_hipcc(), *HIPCC_FLAGS, "-x", "hip", "-c", os.path.join(CSRC, src), "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{res.stdout}\n{res.stderr}")
    return obj


def _compile_marshal() -> str:
    import torch
    from torch.utils.cpp_extension import TORCH_LIB_PATH, include_paths
    paths = [flag for path in include_paths() for flag in ("-isystem", path)]
    cmd = [shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DDT_TORCH_VERSION="{torch.__version__}"',
           "-I", sysconfig.get_path("include"), *paths,
           os.path.join(CSRC, "marshal.cpp"), "-L", TORCH_LIB_PATH, "-ltorch_python", "-o", MARSHAL + ".tmp"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed for marshal.cpp:\n{res.stdout}\n{res.stderr}")
    os.replace(MARSHAL + ".tmp", MARSHAL)
    return MARSHAL


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as pool:
        marshal = pool.submit(_compile_marshal)
        objs = list(pool.map(_compile, SOURCES))
    tmp = LIBRARY + ".tmp"
    cmd = [_hipcc(), "-shared", "-fPIC", f"--offload-arch={ARCH}", *objs, "-o", tmp]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIBRARY)
    marshal.result()  # the library is in place where the helper cannot be built
    if verbose:
        print(f"built {LIBRARY} and {MARSHAL}")
    return LIBRARY


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
