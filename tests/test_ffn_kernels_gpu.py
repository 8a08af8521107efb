"""The GEMM with a residual of the operands' type on every kernel, whole tiles
whose residual is staged in LDS among them, out of place and in place; and the
backward at extents that run the tile shapes which test_ffn_plans_gpu.py leaves
out.  test_ffn_kernels_cpu.py checks that the extents reach them all."""
import pytest
import torch

import ffn_reference as ref
import mlp_megakernel_amd as mk
from helpers import progress
from test_ffn_gpu import problem, rows
from test_ffn_plans_gpu import FORWARD

pytestmark = pytest.mark.gpu

RESIDUAL = FORWARD + [(680, 18124, 141), (7987, 11272, 130), (513, 772, 1032)]
BACKWARD = [(812, 71, 10876), (4850, 526, 4400), (1450, 851, 4308), (3873, 9971, 336), (524, 134, 17195)]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shape", RESIDUAL, ids=str)
def test_residual_of_the_same_type(dt, shape):
    M, N, K = shape
    gen, A, (B,), (b,) = problem(M, N, K, dt)
    R = rows(gen, M, N, 1.0, dt, pad=8)
    Y, Z = mk.gemm_residual_train(A, B, R, b, act="silu")
    v, e, z = ref.residual(A, B, b, R, "silu", dt)
    ref.check(Y, (v, e), "Y")
    ref.check(Z, z, "Z")
    assert torch.equal(mk.gemm_residual(A, B, R, b, act="silu"), Y)
    ld = R.stride(0) if M > 1 else (N + 15) // 8 * 8
    own = torch.full((M, ld), 7.0, dtype=dt, device="cuda")
    own[:, :N] = R
    assert torch.equal(mk.gemm_residual(A, B, own[:, :N], b, act="silu", out=own[:, :N]), Y)
    assert bool((own[:, N:] == 7.0).all())
    # neither activation nor bias, the block's second product
    Y = mk.gemm_residual(A, B, R)
    v, e, _ = ref.residual(A, B, None, R, "none", dt)
    ref.check(Y, (v, e), "Y, no activation")
    progress("residual %s %s" % (dt, shape))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shape", BACKWARD, ids=str)
def test_backward(dt, shape):
    M, N, K = shape
    gen, A, Bs, bs = problem(M, N, K, dt, nb=2)
    _, Z = mk.gated_gemm_train(A, *Bs, *bs, act="gelu")
    dY = rows(gen, M, N, 1.0, dt)
    for grad in (dt, torch.float32):
        g = mk.gated_gemm_backward(A, *Bs, Z, dY, act="gelu", want_dbias=True, grad_dtype=grad)
        r = ref.backward(A, Bs, Z, dY, "gelu", grad)
        for name, got, want in (("dA", g.dA, r["dA"]), ("dBg", g.dBg, r["dB"][0]), ("dBu", g.dBu, r["dB"][1]),
                                ("dbias_g", g.dbias_g, r["dbias"][0]), ("dbias_u", g.dbias_u, r["dbias"][1])):
            ref.check(got, want, name)
        g = mk.gemm_residual_backward(A, Bs[0], dY, Z[0], act="gelu", want_dbias=True, grad_dtype=grad)
        r = ref.backward(A, Bs[:1], Z[:1], dY, "gelu", grad)
        for name, got, want in (("dA", g.dA, r["dA"]), ("dB", g.dB, r["dB"][0]), ("dbias", g.dbias, r["dbias"][0])):
            ref.check(got, want, name)
    progress("backward %s %s" % (dt, shape))
