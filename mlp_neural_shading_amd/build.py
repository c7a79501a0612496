"""Build the HIP library ``libmlp.so`` in-tree with hipcc for gfx950, and the torch form's extension with g++.

Usage: ``python -m mlp_neural_shading_amd.build`` (or ``__graft_entry__.build()``).
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor
from pathlib import Path

PKG = Path(__file__).resolve().parent
CSRC = PKG / "csrc"
LIB = PKG / "libmlp.so"
BUILD_DIR = PKG.parent / "_build"

ARCH = "gfx950"
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
COMMON = [
    "-O3", "-std=c++17", "-fPIC", "-Wall", "-Wno-unused-function",
    # no packed-FP32 instructions anywhere (hipcc's host pass warns that it does not know the feature)
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # a single-lane LDS atomic claims the next tile and its result is read an iteration later; the
    # wave-aggregating rewrite of atomics would consume the result at once and stall the wave
    "-mllvm", "-amdgpu-atomic-optimizer-strategy=None",
]
SOURCES = ["mlp_kernels.hip", "mlp_kernels_fp8.hip", "mlp_layered.hip", "mlp_pack_device.hip", "mlp_api.cpp", "mlp_pack.cpp",
           "mlp_ops_product.hip", "mlp_ops_route.hip", "mlp_ops_api.cpp", "mlp_ops_norm.hip", "mlp_ops_fp8.hip",
           "mlp_ops_fp8_api.cpp"]
CEILING_SOURCE = "mlp_ceiling.hip"
CEILING_LIB = PKG / "libmlp_ceiling.so"

TORCH_SOURCE = "mlp_torch_fp8.cpp"  # the torch form's usual call as a Python extension
TORCH_LIB = PKG / "_torch_fp8.so"


INCLUDE = PKG.parent / "include"


def _compile(src: Path, obj: Path, extra) -> None:
    cmd = [HIPCC, "--offload-arch=" + ARCH, *COMMON, "-I", str(INCLUDE), *extra, "-x", "hip", "-c", str(src),
           "-o", str(obj)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("hipcc failed for %s:\n%s\n%s" % (src.name, " ".join(cmd), r.stderr[-8000:]))


def _compile_torch(obj: Path) -> None:
    import torch
    from sysconfig import get_paths

    at = Path(torch.__file__).parent / "include"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI, "-I", str(INCLUDE), "-isystem", str(at), "-isystem",
           str(at / "torch" / "csrc" / "api" / "include"), "-isystem", "/opt/rocm/include", "-isystem", get_paths()["include"], "-c",
           str(CSRC / TORCH_SOURCE), "-o", str(obj)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed for %s:\n%s\n%s" % (TORCH_SOURCE, " ".join(cmd), r.stderr[-8000:]))


def _link_torch(obj: Path) -> None:
    import torch

    libs = Path(torch.__file__).parent / "lib"
    tmp = TORCH_LIB.with_name(TORCH_LIB.name + ".tmp%d" % os.getpid())
    cmd = ["g++", "-shared", "-fPIC", str(obj), "-o", str(tmp), "-L", str(libs), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_hip",
           "-lc10", "-lc10_hip", "-L", str(PKG), "-l:" + LIB.name, "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (" ".join(cmd), r.stderr[-8000:]))
    os.replace(tmp, TORCH_LIB)


def _no_torch() -> str:
    """Why the extension cannot be built here; empty if it can."""
    if importlib.util.find_spec("torch") is None:
        return "torch is not installed"
    return "" if shutil.which("g++") else "g++ is not installed"


def _link(objs, lib: Path) -> None:
    tmp = lib.with_name(lib.name + ".tmp%d" % os.getpid())
    cmd = [HIPCC, "--offload-arch=" + ARCH, "-shared", "-fPIC", *map(str, objs), "-o", str(tmp)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (" ".join(cmd), r.stderr[-8000:]))
    os.replace(tmp, lib)


def build(verbose: bool = False, extra=()) -> Path:
    """The library and the ceiling probe, which need hipcc alone, and last the extension, which needs torch and g++ too: without
    them it is left out, which is said, and where it does not compile, the others stand."""
    BUILD_DIR.mkdir(exist_ok=True)
    objs = [BUILD_DIR / (Path(s).stem + ".o") for s in SOURCES]
    torch_obj, probe_obj = BUILD_DIR / "mlp_torch_fp8.o", BUILD_DIR / "mlp_ceiling.o"
    missing = _no_torch()
    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        extension = None if missing else ex.submit(_compile_torch, torch_obj)
        list(ex.map(lambda so: _compile(CSRC / so[0], so[1], list(extra)), zip(SOURCES, objs)))
    _link(objs, LIB)
    # the benchmark's MFMA-ceiling probe, a separate small library
    _compile(CSRC / CEILING_SOURCE, probe_obj, list(extra))
    _link([probe_obj], CEILING_LIB)
    TORCH_LIB.unlink(missing_ok=True)  # one of another build may have other structs
    if missing:
        print("%s is left out, and calls of ops_fp8 take some microseconds more: %s" % (TORCH_LIB.name, missing), file=sys.stderr)
    else:
        extension.result()
        _link_torch(torch_obj)
    if verbose:
        print("built %s" % ", ".join(str(p) for p in (LIB, CEILING_LIB, TORCH_LIB) if p.exists()))
    return LIB


if __name__ == "__main__":
    build(verbose=True, extra=sys.argv[1:])
