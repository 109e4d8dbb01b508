"""Build libmnb.so for gfx950 in-tree.

hipcc compiles the kernels (mnb_gemv.hip, mnb_gemv_mfma4.hip,
mnb_gemm_mfma.hip, mnb_layout.hip, mnb_int8.hip, mnb_moe.hip,
mnb_append.hip, mnb_attention.hip, mnb_lora.hip); the host front end
(mnb_api.cpp) is plain C++ built with g++; hipcc links both into one shared
library next to this file.  mnb_torch.cpp, the part of the Python binding that is
compiled, becomes a module of its own there; it alone needs torch and Python's
headers, and where it cannot be built the library is there without it.
"""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmnb.so")
PROBE_LIB = os.path.join(HERE, "libmnb_probe.so")
TORCH_MODULE = os.path.join(HERE, "mnb_torch.so")
ARCH = "gfx950"

HIP_FLAGS = [
    "--offload-arch=" + ARCH, "-O3", "-std=c++17", "-fPIC",
    # no packed-fp32 instructions anywhere in the device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-I", INCLUDE, "-I", CSRC,
]
CXX_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-Wall", "-Wextra", "-I", INCLUDE,
             "-I", CSRC]


def _torch_flags():
    """Compiler and linker flags of the binding's module, which uses torch's
    tensors (no GPU code)."""
    import sysconfig
    import torch
    root = os.path.dirname(torch.__file__)
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    include = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"]]
    # (torch's headers warn under -Wextra)
    flags = ["-O2", "-std=c++17", "-fPIC", "-Wall", "-D_GLIBCXX_USE_CXX11_ABI=%d" % abi, "-I", INCLUDE]
    for path in include:
        flags += ["-isystem", path]
    return flags, ["-L" + os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)


def _build_module(verbose):
    """Compile mnb_torch.so; returns why there is none, or None.  One of older
    sources does not stay."""
    tmp = TORCH_MODULE + ".tmp%d" % os.getpid()
    try:
        flags, libs = _torch_flags()
        _run(["g++", "-shared", os.path.join(CSRC, "mnb_torch.cpp"), "-o", tmp] + flags + libs, verbose)
        os.replace(tmp, TORCH_MODULE)
        return None
    except (ImportError, subprocess.CalledProcessError) as e:
        for path in (tmp, TORCH_MODULE):
            if os.path.exists(path):
                os.remove(path)
        return str(e)


def build(verbose: bool = False, save_temps: bool = False) -> str:
    """Compile and link libmnb.so (always recompiles), and the binding's module
    where torch is there. Returns the library's path."""
    os.makedirs(BUILD, exist_ok=True)
    extra = ["-save-temps=obj"] if save_temps else []
    objs = []
    jobs = []
    for name in ("mnb_gemv", "mnb_gemv_mfma4", "mnb_gemm_mfma", "mnb_layout", "mnb_int8", "mnb_moe",
                 "mnb_append", "mnb_attention", "mnb_lora"):
        obj = os.path.join(BUILD, name + ".o")
        objs.append(obj)
        jobs.append(["hipcc", "-c", os.path.join(CSRC, name + ".hip"), "-o", obj]
                    + HIP_FLAGS + extra)
    api_o = os.path.join(BUILD, "mnb_api.o")
    objs.append(api_o)
    jobs.append(["g++", "-c", os.path.join(CSRC, "mnb_api.cpp"), "-o", api_o] + CXX_FLAGS)
    # The translation units are independent: compile them side by side.
    from concurrent.futures import ThreadPoolExecutor
    with ThreadPoolExecutor(max_workers=len(jobs) + 1) as ex:
        module = ex.submit(_build_module, verbose)
        for f in [ex.submit(_run, cmd, verbose) for cmd in jobs]:
            f.result()
    tmp = LIB + ".tmp%d" % os.getpid()
    _run(["hipcc", "-shared", "-fPIC", "--offload-arch=" + ARCH, "-o", tmp] + objs, verbose)
    os.replace(tmp, LIB)
    # measurement support: read-only HBM streaming probe (bench only)
    tmp = PROBE_LIB + ".tmp%d" % os.getpid()
    _run(["hipcc", "-shared", os.path.join(CSRC, "mnb_probe.hip"), "-o", tmp] + HIP_FLAGS,
         verbose)
    os.replace(tmp, PROBE_LIB)
    why = module.result()
    if why:
        print("mnb_torch.so (append_kv_int8, attention_int8 and matmul_lora from Python) is not built: " + why,
              file=sys.stderr, flush=True)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
