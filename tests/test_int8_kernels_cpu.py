"""The extents of the GPU test of the same name against the plans that they run
(ffn_plan.hpp, compiled here for the host, with the 256 compute units of an
MI355X): together they reach every kernel that a plan of an 8-bit product can
name, each of them once."""
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

PROGRAM = r"""
#include <cstdio>
#include "ffn_plan.hpp"
using namespace coalesce;
int main(int n, char** v) {
  for (int i = 1; i < n; ++i) {
    int gated;
    long M, N, K;
    if (std::sscanf(v[i], "%d:%ld,%ld,%ld", &gated, &M, &N, &K) != 4) return 1;
    const Int8Plan f = plan_int8(M, N, K, gated, 256);
    if (f.few)
      std::printf("few %d\n", (int)f.few);
    else
      std::printf("tile %d%s\n", f.tiles.variant, f.tiles.splits > 1 ? " split" : "");
  }
}
"""


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    cxx = shutil.which(os.environ.get("CXX") or "g++")
    rocm = os.environ.get("ROCM_PATH") or "/opt/rocm"
    if cxx is None or not os.path.exists(os.path.join(rocm, "include", "hip")):
        pytest.skip("no host compiler or no HIP headers")
    d = tmp_path_factory.mktemp("plans8")
    src, exe = d / "plans.cpp", d / "plans"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-O1", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(rocm, "include"),
                    "-I", os.path.join(ROOT, "mlp_megakernel_amd", "csrc"), str(src), "-o", str(exe)], check=True)

    def run(gated, extents):
        args = ["%d:%d,%d,%d" % (gated, *e) for e in extents]
        return subprocess.run([str(exe)] + args, check=True, stdout=subprocess.PIPE, text=True).stdout.splitlines()
    return run


def wanted(few, whole, split):
    return ["few %d" % f for f in few] + ["tile %d" % v for v in whole] + ["tile %d split" % v for v in split]


def test_every_kernel_is_run(plans):
    import test_int8_kernels_gpu as t
    # FEW8_8_LONG (2) is of gated products alone, FEW8_8_WIDE (1) of plain ones; the
    # gated product has no three-stage tiles (7, 8)
    assert sorted(plans(0, t.FEW + t.TILES)) == sorted(wanted((1, 3, 4, 5, 6, 7, 8, 9), range(1, 9), (2, 3, 8)))
    assert sorted(plans(1, t.FEW_GATED + t.TILES_GATED)) == sorted(wanted(range(2, 10), range(1, 7), (2, 3)))


def test_one_row_more_than_the_few(plans):
    assert plans(0, [(64, 40, 40), (65, 40, 40)]) == plans(1, [(64, 40, 40), (65, 40, 40)]) == ["few 8", "tile 3"]
