"""Compile the HIP library ``libdbs.so`` for gfx950 with hipcc, and the binding's compiled part with the host compiler.

Run ``python -m spmspv_graph_traversal_amd.build_lib`` (the repository's
``build()`` calls :func:`build`).  Objects go to ``_build/`` next to this file,
the shared library next to the Python binding.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libdbs.so")
CALLS = os.path.join(HERE, "_calls.so")  # argument marshalling of the decode-step calls (csrc/calls.cpp)
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

SOURCES = ["scan.hip", "build.hip", "spmspv.hip", "bfs.hip", "probe.hip", "q4.hip", "q4_bf16.hip", "q4_bf16_gated.hip",
           "q4_f32.hip", "q4_f32_gated.hip", "logits.hip", "rope.hip", "norm_rope.hip",
           "kv4.hip", "kv4_64.hip", "kv4_96.hip", "kv4_128.hip", "kv4_192.hip", "kv4_256.hip",
           "api.cpp"]

FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-fPIC",
    "-std=c++17",
    "-munsafe-fp-atomics",
    # code objects the HIP runtime bundled with PyTorch can load
    "-mcode-object-version=5",
    "-Wall",
    "-Wno-unused-function",
    # packed fp32 instructions stay off on this target
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def _compile(src: str) -> str:
    obj = os.path.join(OUT_DIR, os.path.basename(src) + ".o")
    cmd = [HIPCC, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    if src.endswith(".cpp"):
        cmd = [HIPCC, *FLAGS, "-x", "hip", "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def rocm_include() -> str:
    """Where HIP's headers are: beside the compiler, which may be named without its folder, or where ROCM_PATH or the usual
    place has them."""
    found = shutil.which(HIPCC)
    for rocm in (os.path.dirname(os.path.dirname(os.path.abspath(found))) if found else None, os.environ.get("ROCM_PATH"), "/opt/rocm"):
        if rocm and os.path.exists(os.path.join(rocm, "include", "hip", "hip_runtime.h")):
            return os.path.join(rocm, "include")
    raise RuntimeError(f"HIP's headers were not found beside {HIPCC}, in ROCM_PATH or in /opt/rocm")


def _compile_calls() -> None:
    import sysconfig

    import torch

    at = os.path.dirname(torch.__file__)
    tmp = CALLS + ".tmp"
    # the macros tell torch's headers which device backend it was built with
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM",
           "-I" + os.path.join(at, "include"), "-I" + os.path.join(at, "include", "torch", "csrc", "api", "include"),
           "-I" + rocm_include(), "-I" + sysconfig.get_paths()["include"],
           os.path.join(CSRC, "calls.cpp"), "-o", tmp, "-L" + os.path.join(at, "lib"),
           "-ltorch_python", "-ltorch_cpu", "-lc10_hip", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"calls.cpp failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALLS)


def build(verbose: bool = False) -> str:
    os.makedirs(OUT_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(len(SOURCES) + 1, os.cpu_count() or 4)) as ex:
        calls = ex.submit(_compile_calls)
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-mcode-object-version=5", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    calls.result()  # after the library, which works without it but for the decode-step calls
    if verbose:
        print(f"built {LIB} and {CALLS}")
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
