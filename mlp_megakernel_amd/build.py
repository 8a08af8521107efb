"""Build libcoalesce.so (the gfx950 HIP kernels and the C ABI) in-tree with hipcc,
and _marshal.so (the binding's reading of tensor lists) with the host compiler.

    python -m mlp_megakernel_amd.build      # or __graft_entry__.build()

Every call recompiles.  Sources are compiled in parallel, one object each, then
linked into ``mlp_megakernel_amd/libcoalesce.so``.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libcoalesce.so")
MARSHAL = os.path.join(HERE, "_marshal.so")
BUILD_DIR = os.path.join(HERE, "_build")
SOURCES = ["mlp.hip", "mlp_alt.hip", "mlp_small.hip", "mlp_stream.hip", "mlp_bwd.hip", "mlp_bwd_stream.hip",
           "gemm16.hip", "gemm32.hip", "elementwise.hip", "matrix_rate.hip", "weightnorm.hip", "ffn.hip",
           "ffn_gated_bf16.hip", "ffn_gated_f16.hip", "ffn_resid_bf16.hip", "ffn_resid_f16.hip",
           "ffn_bwd_bf16.hip", "ffn_bwd_f16.hip", "gradnorm.hip", "abi.cpp"]
ARCH = "gfx950"


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found; install ROCm or set HIPCC")


def compile_flags():
    return [
        "--offload-arch=" + ARCH,
        "-O3",
        "-std=c++17",
        "-fPIC",
        "-Wall",
        "-Wno-unused-function",
        # packed fp32 VALU forms are kept off for the whole library
        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    ]


def _compile(src: str) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [hipcc()] + compile_flags() + ["-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    out = "\n".join(l for l in r.stdout.splitlines() if "packed-fp32-ops" not in l)
    if r.returncode != 0:
        raise RuntimeError("compilation of %s failed:\n%s" % (src, out))
    if out.strip():
        sys.stderr.write(out + "\n")
    return obj


def _build_marshal() -> None:
    """The Python extension csrc/marshal.cpp, against the torch that is installed."""
    import torch
    from torch.utils.cpp_extension import include_paths
    tmp = MARSHAL + ".tmp%d" % os.getpid()
    cmd = [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI]
    for path in include_paths() + [sysconfig.get_paths()["include"]]:
        cmd += ["-isystem", path]
    cmd += [os.path.join(CSRC, "marshal.cpp"), "-o", tmp, "-L" + os.path.join(os.path.dirname(torch.__file__), "lib"),
            "-ltorch_python", "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if r.returncode != 0:
        raise RuntimeError("compilation of marshal.cpp failed:\n" + r.stdout)
    os.replace(tmp, MARSHAL)


def build(verbose: bool = True) -> str:
    jobs = min(len(SOURCES), max(1, int(os.environ.get("MAX_JOBS", os.cpu_count() or 4))))
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        marshal = ex.submit(_build_marshal)
        objs = list(ex.map(_compile, SOURCES))
        marshal.result()
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [hipcc(), "--offload-arch=" + ARCH, "-shared", "-fPIC", "-o", tmp] + objs
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout)
    os.replace(tmp, LIB)
    if verbose:
        print("built", LIB)
    return LIB


if __name__ == "__main__":
    build()
