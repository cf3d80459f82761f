"""Compile the HIP library libtlrgemm.so in-tree for gfx950.

Usage: python -m hpc_linear_algebra_amd.build   (or call build()).
Every source is compiled with hipcc; device code is built for gfx950 only and
with packed-fp32 instructions disabled (the compiler would otherwise form
v_pk_* fp32 arithmetic from ordinary float code).  binding.cpp, host code against
torch's headers, becomes the extension module _binding beside it; the library
needs neither torch nor that module, and is built first.
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
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libtlrgemm.so")
SOURCES = ["planner.cpp", "abi.cpp", "executor.cpp", "noalloc.cpp", "gemm.hip", "gemm16.hip", "compress.hip",
           "block.hip", "moe.hip", "int8.hip", "experts.hip", "gated.hip"]
ARCH = "gfx950"
BINDING = os.path.join(PKG, "_binding" + sysconfig.get_config_var("EXT_SUFFIX"))


def hipcc() -> str:
    cand = os.environ.get("HIPCC") or shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    return cand


def _flags():
    return ["-O3", "-fPIC", "-std=c++17", f"--offload-arch={ARCH}",
            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
            "-Wall", "-Wno-unused-function", "-I", INCLUDE, "-I", CSRC]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [hipcc()] + _flags() + ["-c", os.path.join(CSRC, src), "-o", obj]
    if src.endswith(".cpp"):
        cmd = [hipcc()] + ["-x", "hip"] + _flags() + ["-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    noise = "is not a recognized feature for this target"
    err = "\n".join(l for l in (r.stdout + r.stderr).splitlines() if noise not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{err}")
    if err.strip():
        sys.stderr.write(err + "\n")
    return obj


def _build_binding() -> str:
    import torch
    from torch.utils import cpp_extension
    tmp = BINDING + ".tmp"
    cmd = [hipcc(), "-O2", "-fPIC", "-shared", "-std=c++17", "-Wall", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
           "-isystem", sysconfig.get_paths()["include"]]
    for path in cpp_extension.include_paths("cuda"):
        cmd += ["-isystem", path]
    cmd += ["-x", "c++", os.path.join(CSRC, "binding.cpp"), "-o", tmp]
    cmd += [f"-L{path}" for path in cpp_extension.library_paths("cuda")]
    cmd += ["-lc10", "-lc10_hip", "-ltorch", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("hipcc failed for binding.cpp:\n" + r.stdout + r.stderr)
    os.replace(tmp, BINDING)
    return BINDING


def build(verbose: bool = False) -> str:
    """Compile every source and link libtlrgemm.so and _binding next to this file.
    Without torch the library alone; an extension that does not compile is an
    error, with the library in place."""
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(max_workers=5) as ex:
        binding = ex.submit(_build_binding)
        objs = list(ex.map(_compile, SOURCES))
        tmp = LIB + ".tmp"
        cmd = [hipcc(), "-shared", "-fPIC", f"--offload-arch={ARCH}", "-o", tmp] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
        os.replace(tmp, LIB)
        if verbose:
            print("built", LIB)
        try:
            binding.result()
        except ImportError as e:
            sys.stderr.write(f"{os.path.basename(BINDING)} is not built, it needs torch: {e}\n")
    return LIB


if __name__ == "__main__":
    build(verbose=True)
