"""Build the gfx950 HIP library in-tree (hipcc, no JIT cache)."""
from __future__ import annotations

import os
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_DIR = os.path.join(PKG, "_lib")
LIB_PATH = os.path.join(LIB_DIR, "libmamba_scan.so")
MARSHAL_PATH = os.path.join(LIB_DIR, "mamba_marshal.so")
SOURCES = [os.path.join(CSRC, f) for f in ("mamba_scan.hip", "mamba_scan_ts.hip",
                                            "mamba_scan_bwd.hip", "mamba_gemm.hip",
                                            "mamba_block.hip", "mamba_norm.hip", "mamba_delta.hip",
                                            "mamba_delta_step.hip", "mamba_delta_bwd.hip")]

HIPCC_FLAGS = [
    "-O3", "--offload-arch=gfx950", "-std=c++17", "-fPIC", "-shared",
    # packed fp32 VALU ops (v_pk_*_f32) stay disabled on this target
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
]


def hipcc() -> str:
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    return os.path.join(rocm, "bin", "hipcc")


def build_marshal() -> str:
    """Compile the binding's per-call part (host code only) against torch's headers and the library."""
    import sysconfig

    import torch
    torch_dir = os.path.dirname(torch.__file__)
    tmp = MARSHAL_PATH + ".tmp%d" % os.getpid()
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-w",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI),
           '-DMAMBA_TORCH_VERSION="%s"' % torch.__version__,
           "-I", INCLUDE, "-I", os.path.join(torch_dir, "include"),
           "-I", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], os.path.join(CSRC, "mamba_marshal.cpp"),
           "-o", tmp, "-L", LIB_DIR, "-l:libmamba_scan.so", "-Wl,-rpath,$ORIGIN",
           "-L", os.path.join(torch_dir, "lib"), "-Wl,--no-as-needed", "-ltorch_python", "-ltorch_cpu",
           "-lc10"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("g++ failed:\n" + res.stdout + res.stderr)
    os.replace(tmp, MARSHAL_PATH)
    return MARSHAL_PATH


def build(verbose: bool = False) -> str:
    """Compile every HIP source into selective_state_space_47_amd/_lib/libmamba_scan.so, and the
    binding's per-call part beside it."""
    os.makedirs(LIB_DIR, exist_ok=True)
    tmp = LIB_PATH + ".tmp%d" % os.getpid()
    cmd = [hipcc()] + HIPCC_FLAGS + ["-I", INCLUDE, "-o", tmp] + SOURCES
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + res.stdout + res.stderr)
    if verbose and res.stderr:
        print(res.stderr)
    os.replace(tmp, LIB_PATH)
    build_marshal()
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose=True))
