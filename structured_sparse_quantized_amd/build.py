"""Build the gfx950 HIP library ``libss.so`` and its Python binding ``_ssbind.so`` in place (no JIT cache)."""
from __future__ import annotations

import os
import shutil
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libss.so")
BIND = os.path.join(PKG, "_ssbind.so")
SOURCES = ["ss_api.hip", "k_quant_lift.hip", "k_prune.hip", "k_slide.hip", "k_spgemm.hip", "k_spgemm_tiled.hip",
           "k_spgemm_wide.hip", "k_spgemm_small.hip", "k_quant_spgemm.hip", "k_rotary.hip",
           "k_attn.hip"]

ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
HIPCC = os.environ.get("HIPCC", os.path.join(ROCM, "bin", "hipcc"))
CXX = os.environ.get("CXX", "g++")
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    # no fused multiply-add contraction: every float32 step rounds once
    "-ffp-contract=off",
    # keep packed-fp32 instructions out of the generated code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", INCLUDE, "-I", CSRC,
]


def _run(cmd, what, verbose):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what}:\n{r.stderr}")
    if verbose:
        print(" ".join(cmd))


def _bind_object(objdir, verbose):
    """The binding is host code against torch's headers (the host compiler, no device code)."""
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    obj = os.path.join(objdir, "ss_bind.o")
    _run([CXX, "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
          "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem",
          sysconfig.get_paths()["include"], "-isystem", os.path.join(ROCM, "include"), "-D__HIP_PLATFORM_AMD__", "-c", os.path.join(CSRC, "ss_bind.cpp"), "-o", obj],
         "the host compiler failed for ss_bind.cpp", verbose)
    return obj


def _link_bind(obj, verbose):
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BIND + ".tmp"
    _run([CXX, "-shared", "-fPIC", obj, "-o", tmp, "-L", PKG, "-l:libss.so", "-Wl,-rpath,$ORIGIN", "-L", lib,
          "-ltorch_python", "-ltorch_cpu", "-lc10_hip", "-lc10", f"-Wl,-rpath,{lib}"], "linking _ssbind.so failed", verbose)
    os.replace(tmp, BIND)


def build(verbose: bool = False) -> str:
    """Compile every source for gfx950, link ``libss.so`` and the binding; returns the library's path."""
    objdir = os.path.join(PKG, "_build")
    os.makedirs(objdir, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(objdir, src.replace(".hip", ".o"))
        cmd = [HIPCC, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"hipcc failed for {src}:\n{r.stderr}")
        if verbose:
            print(" ".join(cmd))
        return obj

    with ThreadPoolExecutor(max_workers=8) as ex:
        bind = ex.submit(_bind_object, objdir, verbose)
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    _link_bind(bind.result(), verbose)
    shutil.rmtree(objdir, ignore_errors=True)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
