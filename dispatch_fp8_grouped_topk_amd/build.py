"""Build libmegamoe.so (all HIP sources of csrc/) for gfx950 with hipcc, in place, and the compiled
part of the Python binding, _binding.so (csrc/mm_binding.cpp, host code against torch's headers).

    python -m dispatch_fp8_grouped_topk_amd.build                   # both
    python -m dispatch_fp8_grouped_topk_amd.build --library-only    # the C library, which needs no torch

Compiles every translation unit in parallel into _build/ and links the shared libraries
next to this file.  Always recompiles (it is the package's "does it build" check).
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmegamoe.so")
BINDING = os.path.join(HERE, "_binding.so")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-fvisibility=hidden",
    # no packed-FP32 instructions anywhere in the device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # MFMA results in arch VGPRs: the FP8 recipe promotes every MFMA result with VALU FMAs,
    # which cannot read AGPRs directly
    "-mllvm", "-amdgpu-mfma-vgpr-form",
    "-I", os.path.join(ROOT, "include"), "-I", CSRC,
    "-Wno-unused-command-line-argument",
]


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".hip"))


def _compile(src):
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [HIPCC, *FLAGS, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stderr}")
    return obj


def _compile_binding():
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths
    obj = os.path.join(BUILD, "mm_binding.cpp.o")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-w",
           "-D__HIP_PLATFORM_AMD__", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", os.path.join(ROOT, "include"),
           *[a for d in [*include_paths("cuda"), sysconfig.get_paths()["include"]] for a in ("-isystem", d)],
           "-c", os.path.join(CSRC, "mm_binding.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compiling the binding failed:\n{r.stderr}")
    return obj, os.path.join(os.path.dirname(torch.__file__), "lib")


def _link_binding(obj, torch_lib):
    tmp = BINDING + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-fPIC", obj, "-L", HERE, "-lmegamoe", "-L", torch_lib, "-lc10", "-lc10_hip",
           "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN", "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"linking the binding failed:\n{r.stderr}")
    os.replace(tmp, BINDING)


def build(verbose: bool = True, binding: bool = True) -> str:
    """The C library, with `binding` the compiled part of the Python binding too (torch's headers, a host C++ compiler).
    The library is in place before a failure of the binding is raised."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs) + 1)) as ex:
        bound = ex.submit(_compile_binding) if binding else None
        objs = list(ex.map(_compile, srcs))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    if bound is not None:
        _link_binding(*bound.result())
    if verbose:
        print(f"built {LIB} from {len(srcs)} sources", file=sys.stderr)
    return LIB


if __name__ == "__main__":
    if sys.argv[1:] not in ([], ["--library-only"]):
        sys.exit("usage: build [--library-only]")
    build(binding=not sys.argv[1:])
