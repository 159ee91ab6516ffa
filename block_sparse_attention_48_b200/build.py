"""Build the CUDA library (libflexattn.so) in-tree with nvcc for sm_100a, and the Python
binding of the serving calls (_binding.so) with g++ against torch's headers.

    python block_sparse_attention_48_b200/build.py [--force] [--verbose]

The library exports the C ABI declared in include/flexattn.h.
"""

from __future__ import annotations

import argparse
import concurrent.futures
import glob
import importlib.util
import os
import re
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libflexattn.so")
BUILD_DIR = os.path.join(PKG, "_build")
BINDING = os.path.join(PKG, "_binding.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
    "--expt-relaxed-constexpr",
]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale() -> bool:
    return _older(LIB, sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) +
                  glob.glob(os.path.join(INCLUDE, "*.h")))


def _older(target: str, deps) -> bool:
    return not os.path.exists(target) or any(os.path.getmtime(d) > os.path.getmtime(target) for d in deps)


def _torch() -> tuple:
    """(directory, version) of the installed torch, without importing it."""
    where = importlib.util.find_spec("torch").submodule_search_locations[0]
    with open(os.path.join(where, "version.py")) as f:
        return where, re.search(r"__version__[^=\n]*=\s*['\"]([^'\"]+)", f.read()).group(1)


def build_binding(force: bool = False) -> str:
    """Compile _binding.so (no CUDA code).  It is good for the torch and the Python that it
    was built against, which _build/_binding.for names."""
    torch_dir, version = _torch()
    built_for, record = f"torch {version}, {sysconfig.get_config_var('SOABI')}", os.path.join(BUILD_DIR, "_binding.for")
    if not force and not _older(BINDING, [BINDING_SRC] + glob.glob(os.path.join(INCLUDE, "*.h"))):
        if os.path.exists(record):
            with open(record) as f:
                if f.read() == built_for:
                    return BINDING
    inc, lib = os.path.join(torch_dir, "include"), os.path.join(torch_dir, "lib")
    cuda = os.path.dirname(os.path.dirname(nvcc())) or "/usr/local/cuda"
    tmp = BINDING + f".tmp{os.getpid()}"
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-Wall", f'-DFA_TORCH_VERSION="{version}"',
                           "-I", INCLUDE, "-isystem", inc,
                           "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
                           "-isystem", os.path.join(cuda, "include"), "-isystem", sysconfig.get_paths()["include"],
                           BINDING_SRC, "-o", tmp, "-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"])
    os.replace(tmp, BINDING)
    os.makedirs(BUILD_DIR, exist_ok=True)
    with open(record, "w") as f:
        f.write(built_for)
    return BINDING


def build(force: bool = False, verbose: bool = False) -> str:
    build_binding(force)
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    objs, cmds = [], []
    for src in sources():
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [nvcc(), *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
        if verbose:
            cmd += ["-Xptxas", "-v"]
        cmds.append(cmd)
        objs.append(obj)
    # one nvcc per source file, in parallel
    with concurrent.futures.ThreadPoolExecutor(max_workers=max(1, min(len(cmds), os.cpu_count() or 1))) as ex:
        for f in [ex.submit(subprocess.check_call, c) for c in cmds]:
            f.result()
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.check_call([nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", tmp, *objs])
    os.replace(tmp, LIB)
    return LIB


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    a = ap.parse_args(argv)
    print(build(force=a.force, verbose=a.verbose))


if __name__ == "__main__":
    sys.exit(main())
