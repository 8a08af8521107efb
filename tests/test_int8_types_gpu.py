"""Every kernel of the products on 8-bit operands in every type of result: the 16-bit ones
have an end of their own (residuals and rows through LDS, columns ahead, row blocks in
pairs).  The extents are those that reach every kernel with fp32 results."""
import pytest
import torch

import block_reference as ref
import mlp_megakernel_amd as mk
from ffn_reference import U32 as U
from ffn_reference import act_bound
from helpers import progress
from test_int8_gpu import problem, product
from test_int8_kernels_gpu import FEW, FEW_GATED, TILES, TILES_GATED

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.mark.parametrize("extents", FEW + TILES, ids="x".join(["%d"] * 3).__mod__)
def test_plain(extents):
    M, N, K = extents
    gen, A, sa, (B,), (sb,), (bias,) = problem(M, N, K, 1)
    z, ez = product(A, B, sa, sb, bias)
    for out in DT.values():
        progress("int8 %s %s" % (extents, out))
        R = ref.rows(gen, M, N, out, pad=1)
        for act, r in (("gelu", R), ("silu", None)):
            f, ef = act_bound(z, ez, act, False)
            v, e = f, ef + U * f.abs()
            if r is not None:
                v = f + ref.f64(r)
                e = e + U * v.abs()
            Y, untouched = ref.space(M, N, out, pad=1)
            mk.gemm_int8(A, B, sa, sb, bias, r, act, out=Y)
            ref.check(Y, (v, ref.rounded(v, e, out)), "Y of %s" % out)
            assert untouched()
            if r is not None:  # formed in place
                X, untouched = ref.space(M, N, out)
                X.copy_(r)
                assert torch.equal(mk.gemm_int8(A, B, sa, sb, bias, X, act, out=X), Y) and untouched()


@pytest.mark.parametrize("extents", FEW_GATED + TILES_GATED, ids="x".join(["%d"] * 3).__mod__)
def test_gated(extents):
    M, N, K = extents
    _, A, sa, (Bg, Bu), sb, bias = problem(M, N, K, 1, 2)
    (zg, eg), (zu, eu) = product(A, Bg, sa, sb[0], bias[0]), product(A, Bu, sa, sb[1], bias[1])
    for act in ("silu", "gelu"):
        f, ef = act_bound(zg, eg, act, False)
        v = f * zu
        e = f.abs() * eu + zu.abs() * ef + ef * eu + U * v.abs()
        for out in DT.values():
            progress("int8 gated %s %s %s" % (extents, act, out))
            Y, untouched = ref.space(M, N, out, pad=1)
            mk.gated_gemm_int8(A, Bg, Bu, sa, sb[0], sb[1], bias[0], bias[1], act=act, out=Y)
            ref.check(Y, (v, ref.rounded(v, e, out)), "Y of %s" % out)
            assert untouched()
