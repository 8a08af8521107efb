"""Arguments of the entry points around the feed-forward products at the edge of what
they take, checked on the host (fake pointers, never dereferenced)."""
import os
import shutil
import subprocess

import pytest

import mlp_megakernel_amd as mk
from conftest import ROOT
from test_block_abi_cpu import DEV, INV, NORM, _without_gpu, call  # noqa: F401 (the fixture: these need no GPU)


@pytest.mark.parametrize("eps,status", [(0.0, DEV), (1e-50, DEV), (3.4e38, DEV), (3.5e38, INV), (1e300, INV)])
def test_eps_is_a_number_of_fp32(eps, status):
    assert call("coalesce_layer_norm", NORM, dict(eps=eps)) == status


# ---------------------------------------------------------------------------
# What the entry points hand to the launchers: abi_block.cpp, compiled for the
# host, in front of launchers that write their parameters down
# ---------------------------------------------------------------------------

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "abi_check.hpp"
#include "block.hpp"
using namespace coalesce;
extern "C" hipError_t hipGetDevice(int* d) { return *d = 0, hipSuccess; }
extern "C" hipError_t hipDeviceGetAttribute(int* v, hipDeviceAttribute_t, int) { return *v = 256, hipSuccess; }
extern "C" const char* hipGetErrorString(hipError_t) { return ""; }
namespace coalesce {
hipError_t launch_norm(const NormParams&, DType, DType, hipStream_t) { return hipSuccess; }
size_t norm_backward_workspace(int64_t, int64_t, int) { return 0; }
hipError_t launch_norm_backward(NormBwdParams, DType, DType, hipStream_t, int) { return hipSuccess; }
hipError_t launch_dropout(const DropoutParams&, DType, DType, hipStream_t) { return hipSuccess; }
hipError_t launch_quantize_rows(const QuantParams&, DType, hipStream_t) { return hipSuccess; }
hipError_t launch_quantize_columns(const QuantParams&, DType, hipStream_t) { return hipSuccess; }
size_t int8_workspace(int64_t, int64_t, int64_t, bool, int) { return 0; }
hipError_t launch_int8(const Int8Params& p, bool gated, DType, hipStream_t, int, void*) {
  std::printf("%d %lld %lld\n", (int)gated, (long long)p.lda, (long long)p.ldb);
  return hipSuccess;
}
}  // namespace coalesce
int main(int, char** v) {
  const long long M = std::atoll(v[1]), K = std::atoll(v[2]), lda = std::atoll(v[3]), ldb = std::atoll(v[4]);
  auto at = [](int i) { return (void*)(uintptr_t)(i << 20); };
  auto f = [&](int i) { return (const float*)at(i); };
  int8_t* const a = K ? (int8_t*)at(1) : nullptr;
  int8_t* const b = K ? (int8_t*)at(2) : nullptr;
  int8_t* const u = K ? (int8_t*)at(3) : nullptr;
  int s = coalesce_gemm_int8(a, lda, b, ldb, f(4), f(5), nullptr, nullptr, 0, at(6), 64, M, 64, K, COALESCE_F32,
                             COALESCE_ACT_NONE, nullptr, 0, nullptr);
  s |= coalesce_gated_gemm_int8(a, lda, b, u, ldb, f(4), f(5), f(7), nullptr, nullptr, at(6), 64, M, 64, K, COALESCE_F32,
                                COALESCE_ACT_SILU, nullptr, 0, nullptr);
  return s;
}
"""


@pytest.fixture(scope="module")
def launched(tmp_path_factory):
    cxx = shutil.which(os.environ.get("CXX") or "g++")
    rocm = os.environ.get("ROCM_PATH") or "/opt/rocm"
    if cxx is None or not os.path.exists(os.path.join(rocm, "include", "hip")):
        pytest.skip("no host compiler or no HIP headers")
    d, csrc = tmp_path_factory.mktemp("entry"), os.path.join(ROOT, "mlp_megakernel_amd", "csrc")
    (d / "main.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-O1", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(rocm, "include"), "-I", csrc,
                    str(d / "main.cpp"), os.path.join(csrc, "abi_block.cpp"), "-o", str(d / "entry")], check=True)

    def run(*args):
        return subprocess.run([str(d / "entry"), *map(str, args)], check=True, stdout=subprocess.PIPE,
                              text=True).stdout.splitlines()
    return run


@pytest.mark.parametrize("M", [1, 16, 64, 100])
@pytest.mark.parametrize("ld", [-16, 1, 1 << 30, 1 << 40])
def test_pitches_without_a_contraction_reach_no_kernel(launched, M, ld):
    # A and B have no elements and their pitches are not checked: what addresses memory by them would read anywhere
    assert launched(M, 0, ld, ld) == ["0 0 0", "1 0 0"]


def test_pitches_of_a_contraction_do(launched):
    assert launched(5, 48, 64, 80) == ["0 64 80", "1 64 80"]
