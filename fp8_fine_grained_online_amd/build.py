"""Build libfp8q.so (HIP, gfx950) in-tree with hipcc, and beside it the native part
of the Python binding (host code, against the installed torch). Where torch or
Python's headers are not installed the library is built alone.

Usage: python -m fp8_fine_grained_online_amd.build [--verbose]
"""

import importlib.util
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
BUILD_DIR = os.path.join(PKG_DIR, "_build")
LIB_PATH = os.path.join(PKG_DIR, "libfp8q.so")

SOURCES = ["quant.hip", "retile.hip", "norm.hip", "moe.hip", "gemm.hip", "gemm_qa.hip", "route.hip",
           "tokens.hip", "int8.hip", "norm_rows.hip", "swiglu.hip",
           "ortho.hip", "api.cpp"]
HEADERS = ["common.hpp", "tiles.hpp", "wave.hpp", "rows.hpp"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
FLAGS = [
    "-O3", "-std=c++17", "-fPIC", "-fvisibility=hidden", f"--offload-arch={ARCH}",
    # packed-FP32 VALU forms are disabled for all device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # no implicit multiply-add fusion: every rounding the kernels' arithmetic
    # is specified with happens as written (HIP's header versions of the
    # __fmul_rn/__dmul_rn intrinsics are plain products that would otherwise
    # be contracted into a following addition); FMAs are always explicit
    "-ffp-contract=off",
    "-Wall", "-Wno-unused-command-line-argument",
    "-I", os.path.join(ROOT, "include"),
]


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"command failed ({r.returncode}): {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return r


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, src + ".o")
        lang = ["-x", "hip"] if src.endswith(".hip") else []
        _run([HIPCC, *FLAGS, *lang, "-c", os.path.join(CSRC, src), "-o", obj], verbose)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB_PATH + ".tmp"
    _run([HIPCC, "-shared", "-fPIC", f"--offload-arch={ARCH}", *objs, "-o", tmp], verbose)
    os.replace(tmp, LIB_PATH)
    missing = binding_needs()
    if missing:
        print(f"{missing}: the native part of the binding is not built", file=sys.stderr)
    else:
        build_binding(verbose)
    build_probes(verbose)
    return LIB_PATH


BINDING_PATH = os.path.join(PKG_DIR, "_binding.so")


def binding_needs() -> str:
    """What the binding's native part needs and does not find ('' for nothing)."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        return "torch is not installed"
    for folder, header in ((os.path.join(spec.submodule_search_locations[0], "include"), "ATen/core/Tensor.h"),
                           (sysconfig.get_paths()["include"], "Python.h")):
        if not os.path.exists(os.path.join(folder, header)):
            return f"{os.path.join(folder, header)} is missing"
    return ""


def build_binding(verbose: bool = False) -> str:
    torch_dir = importlib.util.find_spec("torch").submodule_search_locations[0]
    libs = os.path.join(torch_dir, "lib")
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    _run([HIPCC, "-x", "c++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-fvisibility=hidden",
          "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM", "-I", sysconfig.get_paths()["include"],
          "-I", os.path.join(torch_dir, "include"), "-I", os.path.join(rocm, "include"),
          os.path.join(CSRC, "binding.cpp"), "-o", BINDING_PATH + ".tmp",
          "-L", libs, "-ltorch_python", "-ltorch_cpu", "-ltorch_hip", "-lc10", "-lc10_hip",
          "-L", os.path.join(rocm, "lib"), "-lamdhip64", "-L", PKG_DIR, "-l:" + os.path.basename(LIB_PATH),
          "-Wl,-rpath,$ORIGIN"], verbose)
    os.replace(BINDING_PATH + ".tmp", BINDING_PATH)
    return BINDING_PATH


# Test-only GPU probes (tests/probes/*.hip), each built into its own shared
# library next to its source; the product library never loads them.
PROBE_DIR = os.path.join(ROOT, "tests", "probes")


def build_probes(verbose: bool = False):
    if not os.path.isdir(PROBE_DIR):
        return []
    out = []
    for src in sorted(f for f in os.listdir(PROBE_DIR) if f.endswith(".hip")):
        lib = os.path.join(PROBE_DIR, "lib" + src[:-4] + ".so")
        _run([HIPCC, *FLAGS, "-shared", "-x", "hip", os.path.join(PROBE_DIR, src), "-o", lib + ".tmp"],
             verbose)
        os.replace(lib + ".tmp", lib)
        out.append(lib)
    return out


if __name__ == "__main__":
    print(build(verbose="--verbose" in sys.argv))
