"""Parity of the feed-forward operators at extents that run each of their
kernels: every tile shape with and without a split contraction, and the few-row
kernel's strips of 64, 32 and 16 columns for up to 16, 32 and 64 rows (which
kernel runs follows from the extents and the number of compute units; the
extents here reach all of them on 256)."""
import pytest
import torch

import ffn_reference as ref
import mlp_megakernel_amd as mk
from helpers import progress
from test_ffn_gpu import problem, rows

pytestmark = pytest.mark.gpu

FORWARD = [(1, 40, 64), (17, 40, 64), (40, 40, 64), (1, 4100, 64), (17, 4100, 64), (40, 4100, 64), (1, 8200, 72),
           (17, 8200, 64), (63, 8200, 70), (1, 40, 2050), (65, 40, 64), (65, 40, 1001), (65, 200, 64), (3000, 1030, 64),
           (1025, 1030, 4100), (500, 1030, 4100), (1537, 2731, 64), (4100, 5461, 130), (8200, 4100, 130),
           (1537, 4100, 130), (3000, 4100, 130), (500, 8200, 520), (500, 16400, 130), (1537, 2731, 520),
           (2050, 4100, 130), (2050, 520, 4100), (3000, 200, 4100), (1537, 4100, 200), (8192, 4096, 64), (777, 4100, 2050),
           (900, 900, 8200), (900, 1000, 8200)]
BACKWARD = [(1, 40, 64), (777, 40, 64), (40, 200, 64), (1, 40, 130), (65, 40, 130), (500, 4100, 520), (4100, 1030, 200),
            (257, 4100, 1001), (1, 8200, 200), (4100, 40, 1001), (2050, 200, 4100), (3000, 40, 4100), (500, 40, 8200),
            (8200, 40, 4100), (1300, 8200, 200), (4100, 1540, 200), (4100, 2731, 200), (3000, 200, 4100),
            (8192, 72, 4096), (2050, 2731, 520), (3000, 2731, 520), (3000, 2731, 1030), (900, 8200, 1000),
            (8200, 900, 1000), (8200, 500, 1000)]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shape", FORWARD, ids=str)
def test_forward(dt, shape):
    M, N, K = shape
    gen, A, (Bg, Bu), (bg, bu) = problem(M, N, K, dt, nb=2)
    H, (Zg, Zu) = mk.gated_gemm_train(A, Bg, Bu, bg, bu, act="silu")
    v, e, zg, zu = ref.gated(A, Bg, Bu, bg, bu, "silu", dt)
    ref.check(H, (v, e), "H")
    ref.check(Zg, zg, "Zg")
    ref.check(Zu, zu, "Zu")
    R = rows(gen, M, N, 1.0, torch.float32)
    Y, Z = mk.gemm_residual_train(A, Bg, R, bg, act="gelu")
    v, e, z = ref.residual(A, Bg, bg, R, "gelu", torch.float32)
    ref.check(Y, (v, e), "Y")
    ref.check(Z, z, "Z")
    progress("forward %s %s" % (dt, shape))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shape", BACKWARD, ids=str)
def test_backward(dt, shape):
    M, N, K = shape
    gen, A, Bs, bs = problem(M, N, K, dt, nb=2)
    _, Z = mk.gated_gemm_train(A, *Bs, *bs, act="silu")
    dY = rows(gen, M, N, 1.0, dt)
    for grad in (dt, torch.float32):
        g = mk.gated_gemm_backward(A, *Bs, Z, dY, act="silu", want_dbias=True, grad_dtype=grad)
        r = ref.backward(A, Bs, Z, dY, "silu", grad)
        for name, got, want in (("dA", g.dA, r["dA"]), ("dBg", g.dBg, r["dB"][0]), ("dBu", g.dBu, r["dB"][1]),
                                ("dbias_g", g.dbias_g, r["dbias"][0]), ("dbias_u", g.dbias_u, r["dbias"][1])):
            ref.check(got, want, name)
    g = mk.gemm_residual_backward(A, Bs[0], dY, want_dbias=True)
    r = ref.backward(A, Bs[:1], None, dY, "none", torch.float32)
    for name, got, want in (("dA", g.dA, r["dA"]), ("dB", g.dB, r["dB"][0]), ("dbias", g.dbias, r["dbias"][0])):
        ref.check(got, want, name)
    progress("backward %s %s" % (dt, shape))


def test_repeated_calls_give_the_same_bits():
    for (M, N, K) in [(7, 4100, 1001), (500, 1030, 4100), (2050, 200, 4100), (777, 40, 64)]:
        gen, A, Bs, bs = problem(M, N, K, torch.bfloat16, nb=2)
        dY = rows(gen, M, N, 1.0, torch.bfloat16)
        one = two = None
        for _ in range(3):
            H, Z = mk.gated_gemm_train(A, *Bs, *bs)
            g = mk.gated_gemm_backward(A, *Bs, Z, dY, want_dbias=True)
            one, two = two, [H, *Z, *g]
            if one is not None:
                assert all(torch.equal(a, b) for a, b in zip(one, two)), (M, N, K)
