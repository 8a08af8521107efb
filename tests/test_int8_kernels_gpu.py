"""Every kernel of the products on 8-bit operands, at the smallest work that the
choice between them gives it: the forms for few rows, each tile shape with a last
K step that is not whole, whole and split contractions.  Which kernels these
extents reach, the CPU test of the same name shows.
"""
import pytest
import torch

import block_reference as ref
import mlp_megakernel_amd as mk
from ffn_reference import U32 as U
from ffn_reference import act_bound
from helpers import progress
from test_int8_gpu import problem, product

pytestmark = pytest.mark.gpu

# few rows: weights that fit the caches and weights that do not, strips of columns
# once and several times around the compute units
FEW = [(2, 300, 5001), (2, 4500, 301), (14, 100, 300), (21, 130, 333), (40, 100, 385), (37, 4250, 261),
       (1, 8201, 8209), (13, 8201, 8209)]
FEW_GATED = [(2, 300, 5001), (14, 100, 300), (21, 130, 333), (40, 100, 385), (37, 4250, 261), (3, 2567, 13135),
             (2, 8209, 4101), (12, 4134, 8431)]
TILES = [(2112, 6458, 1527), (2955, 1406, 1447), (2757, 469, 18777), (74, 16, 1533), (79, 17, 1625), (969, 10982, 413),
         (6968, 1347, 457), (2375, 3395, 427), (69, 74, 507), (458, 8138, 3755), (2677, 343, 16923)]
TILES_GATED = [(2343, 2974, 1413), (7146, 390, 1417), (4937, 129, 14251), (180, 16, 1401), (74, 16, 1533),
               (1784, 3278, 1455), (6239, 771, 1534), (3532, 1175, 1415)]


@pytest.mark.parametrize("extents", FEW + TILES)
def test_plain(extents):
    M, N, K = extents
    gen, A, sa, (B,), (sb,), (bias,) = problem(M, N, K, 1)
    R = ref.rows(gen, M, N, torch.float32)
    progress("int8 %s" % (extents,))
    Y, untouched = ref.space(M, N, torch.float32, pad=1)
    mk.gemm_int8(A, B, sa, sb, bias, R, "gelu", out=Y)
    z, ez = product(A, B, sa, sb, bias)
    f, ef = act_bound(z, ez, "gelu", False)
    v = f + ref.f64(R)
    ref.check(Y, (v, ef + U * (f.abs() + 2 * v.abs())), "Y")
    assert untouched()
    m = M // 2
    assert torch.equal(mk.gemm_int8(A[m:m + 1], B, sa[m:m + 1], sb, bias, R[m:m + 1], "gelu",
                                    out_dtype=torch.float32), Y[m:m + 1])


@pytest.mark.parametrize("extents", FEW_GATED + TILES_GATED)
def test_gated(extents):
    M, N, K = extents
    _, A, sa, (Bg, Bu), sb, bias = problem(M, N, K, 1, 2)
    progress("int8 gated %s" % (extents,))
    Y, untouched = ref.space(M, N, torch.float32, pad=1)
    mk.gated_gemm_int8(A, Bg, Bu, sa, sb[0], sb[1], bias[0], bias[1], act="silu", out=Y)
    (zg, eg), (zu, eu) = product(A, Bg, sa, sb[0], bias[0]), product(A, Bu, sa, sb[1], bias[1])
    f, ef = act_bound(zg, eg, "silu", False)
    v = f * zu
    e = f.abs() * eu + zu.abs() * ef + ef * eu + U * v.abs()
    ref.check(Y, (v, e + U * v.abs()), "Y")
    assert untouched()
    m = M // 2
    assert torch.equal(mk.gated_gemm_int8(A[m:m + 1], Bg, Bu, sa[m:m + 1], *sb, *bias, act="silu",
                                          out_dtype=torch.float32), Y[m:m + 1])
