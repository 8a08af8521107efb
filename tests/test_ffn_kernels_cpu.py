"""The extents of the GPU tests against the plans that they run (ffn_plan.hpp,
compiled here for the host, with the 256 compute units of an MI355X): together
they reach every kernel that a plan can name."""
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
    char way;
    long M, N, K;
    if (std::sscanf(v[i], "%c:%ld,%ld,%ld", &way, &M, &N, &K) != 4) return 1;
    for (int gated = 0; gated < 2; ++gated) {
      const char* op = gated ? "gated" : "residual";
      auto tile = [&](const char* what, const TilePlan& t) {
        std::printf("%s %s %d%s\n", op, what, t.variant, t.splits > 1 ? " split" : "");
      };
      if (way == 'f') {
        const ForwardPlan f = plan_forward(M, N, K, gated, 256);
        if (f.strip)
          std::printf("%s strip %d rows %d\n", op, f.strip, M <= 16 ? 16 : M <= 32 ? 32 : 64);
        else
          tile("forward", f.tiles);
      } else {
        const BwdPlan b = bwd_plan(M, N, K, gated, 256);
        tile("dA", b.dx);
        tile("dB", b.dw);
      }
    }
  }
}
"""


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    cxx = shutil.which(os.environ.get("CXX") or "g++")
    rocm = os.environ.get("ROCM_PATH") or "/opt/rocm"
    if cxx is None or not os.path.exists(os.path.join(rocm, "include", "hip")):
        pytest.skip("no host compiler or no HIP headers")
    d = tmp_path_factory.mktemp("plans")
    src, exe = d / "plans.cpp", d / "plans"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-O1", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(rocm, "include"),
                    "-I", os.path.join(ROOT, "mlp_megakernel_amd", "csrc"), str(src), "-o", str(exe)], check=True)

    def run(way, extents):
        args = ["%s:%d,%d,%d" % (way, *e) for e in extents]
        return set(subprocess.run([str(exe)] + args, check=True, stdout=subprocess.PIPE, text=True).stdout.splitlines())
    return run


def wanted(op, what, whole, split):
    return {"%s %s %d" % (op, what, v) for v in whole} | {"%s %s %d split" % (op, what, v) for v in split}


def strips(op):
    return {"%s strip %d rows %d" % (op, s, r) for s in (16, 32, 64) for r in (16, 32, 64)}


def test_every_kernel_is_run(plans):
    import test_ffn_kernels_gpu as more
    import test_ffn_plans_gpu as base
    forward = plans("f", base.FORWARD)
    # the gated product has no three-stage shapes, splits run on the 128 x 128 and
    # 64 x 64 ones
    assert {p for p in forward if p.startswith("gated")} == wanted("gated", "forward", range(1, 7), (2, 3)) | strips("gated")
    residual = {p for p in plans("f", more.RESIDUAL) if p.startswith("residual")}
    assert residual == wanted("residual", "forward", range(1, 9), (2, 3, 8)) | strips("residual")
    # A^T dZ has no shapes of 224, 192 and 160 rows
    back = plans("b", base.BACKWARD + more.BACKWARD)
    assert back == set().union(*(wanted(op, "dA", range(1, 9), (2, 3, 8)) | wanted(op, "dB", (1, 2, 3, 7, 8), (2, 3, 8))
                                 for op in ("gated", "residual")))
