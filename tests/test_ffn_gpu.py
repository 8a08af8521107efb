"""GPU parity of the feed-forward operators (gated product, GEMM with residual,
their gradients) with 64-bit references, within bounds derived per element
(ffn_reference.py): odd extents, padded pitches, every type and activation,
empty extents, NaN-filled padding, neighbouring rows left as they were.
"""
import pytest
import torch

import ffn_reference as ref
import mlp_megakernel_amd as mk
from helpers import progress

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
# (M, N, K): single elements and tokens, ragged tails in every extent, several
# tiles, long and short contractions
SHAPES = [(1, 1, 1), (1, 5, 3), (2, 8, 64), (1, 1000, 513), (7, 33, 65), (16, 64, 128), (17, 100, 40), (33, 129, 63),
          (48, 40, 1000), (64, 64, 64), (65, 257, 130), (130, 300, 200), (257, 130, 129), (300, 520, 260),
          (513, 72, 70)]


def rows(gen, m, n, std, dtype, pad=0):
    """m x n ~ N(0, std) in a buffer whose padding (to 16 bytes, and `pad` more
    columns) holds NaN."""
    per = 16 // torch.empty((), dtype=dtype).element_size()
    ld = max(per, (n + per - 1) // per * per) + pad
    t = torch.full((m, ld), float("nan"), dtype=dtype)
    t[:, :n] = (torch.randn(m, n, generator=gen) * std).to(dtype)
    return t.to("cuda")[:, :n]


def vec(gen, n, std, dtype):
    return (torch.randn(n, generator=gen) * std).to(dtype).to("cuda")


def problem(M, N, K, dt, seed=0, pad=0, nb=1):
    gen = torch.Generator().manual_seed(seed + 7919 * M + 104729 * N + K)
    A = rows(gen, M, K, 1.0, dt, pad)
    Bs = [rows(gen, K, N, max(K, 1) ** -0.5, dt, 2 * pad) for _ in range(nb)]
    bs = [vec(gen, N, 0.5, dt) for _ in range(nb)]
    return gen, A, Bs, bs


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("out", ["same", "f32"])
@pytest.mark.parametrize("act", ["silu", "gelu", "relu", "softplus", "none"])
def test_gated_forward(dt, out, act):
    for j, (M, N, K) in enumerate(SHAPES):
        progress("gated %s->%s %s %s" % (dt, out, act, (M, N, K)))
        d = DT[dt]
        od = d if out == "same" else torch.float32
        _, A, (Bg, Bu), (bg, bu) = problem(M, N, K, d, nb=2, pad=8 * (j % 2))
        if j % 3 == 0:
            bg = bu = None
        elif j % 3 == 1:
            bu = None
        H, (Zg, Zu) = mk.gated_gemm_train(A, Bg, Bu, bg, bu, act=act, out_dtype=od)
        H2 = mk.gated_gemm(A, Bg, Bu, bg, bu, act=act, out_dtype=od)
        v, e, zg, zu = ref.gated(A, Bg, Bu, bg, bu, act, od)
        ref.check(H, (v, e), "H %s" % ((M, N, K),))
        ref.check(Zg, zg, "Zg %s" % ((M, N, K),))
        ref.check(Zu, zu, "Zu %s" % ((M, N, K),))
        assert torch.equal(H, H2), "the training forward gives other bits"


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("out", ["same", "f32"])
@pytest.mark.parametrize("act", ["none", "gelu", "silu", "softplus", "relu"])
def test_residual_forward(dt, out, act):
    for j, (M, N, K) in enumerate(SHAPES):
        progress("residual %s->%s %s %s" % (dt, out, act, (M, N, K)))
        d = DT[dt]
        od = d if out == "same" else torch.float32
        gen, A, (B,), (b,) = problem(M, N, K, d, pad=8 * (j % 2))
        R = rows(gen, M, N, 1.0, od, pad=8) if j % 4 else None
        b = b if j % 2 else None
        Y, Z = mk.gemm_residual_train(A, B, R, b, act=act, out_dtype=od)
        v, e, z = ref.residual(A, B, b, R, act, od)
        ref.check(Y, (v, e), "Y %s" % ((M, N, K),))
        ref.check(Z, z, "Z %s" % ((M, N, K),))
        assert torch.equal(Y, mk.gemm_residual(A, B, R, b, act=act, out_dtype=od))
        if R is not None:  # in place: the same bits, the padding untouched
            Rc = torch.full((M, R.stride(0) if M > 1 else (N + 15) // 8 * 8), 7.0, dtype=od, device="cuda")
            Rc[:, :N] = R
            got = mk.gemm_residual(A, B, Rc[:, :N], b, act=act, out=Rc[:, :N])
            assert torch.equal(got, Y) and bool((Rc[:, N:] == 7.0).all())


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("grad", ["same", "f32"])
@pytest.mark.parametrize("act", ["silu", "gelu", "relu", "softplus", "none"])
def test_gated_backward(dt, grad, act):
    for j, (M, N, K) in enumerate(SHAPES):
        progress("gated backward %s %s %s %s" % (dt, grad, act, (M, N, K)))
        d = DT[dt]
        gd = d if grad == "same" else torch.float32
        gen, A, Bs, bs = problem(M, N, K, d, nb=2, pad=8 * (j % 2))
        _, Z = mk.gated_gemm_train(A, *Bs, *bs, act=act)
        dY = rows(gen, M, N, 1.0, torch.float32 if j % 3 == 2 else d, pad=8)
        g = mk.gated_gemm_backward(A, *Bs, Z, dY, act=act, want_dbias=True, grad_dtype=gd)
        r = ref.backward(A, Bs, Z, dY, act, gd)
        ref.check(g.dA, r["dA"], "dA %s" % ((M, N, K),))
        ref.check(g.dBg, r["dB"][0], "dBg %s" % ((M, N, K),))
        ref.check(g.dBu, r["dB"][1], "dBu %s" % ((M, N, K),))
        ref.check(g.dbias_g, r["dbias"][0], "dbias_g %s" % ((M, N, K),))
        ref.check(g.dbias_u, r["dbias"][1], "dbias_u %s" % ((M, N, K),))


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("grad", ["same", "f32"])
@pytest.mark.parametrize("act", ["none", "gelu", "silu", "softplus", "relu"])
def test_residual_backward(dt, grad, act):
    for j, (M, N, K) in enumerate(SHAPES):
        progress("residual backward %s %s %s %s" % (dt, grad, act, (M, N, K)))
        d = DT[dt]
        gd = d if grad == "same" else torch.float32
        gen, A, Bs, bs = problem(M, N, K, d, pad=8 * (j % 2))
        _, Z = mk.gemm_residual_train(A, Bs[0], None, bs[0], act=act)
        dY = rows(gen, M, N, 1.0, torch.float32 if j % 3 == 2 else d, pad=8)
        g = mk.gemm_residual_backward(A, Bs[0], dY, preact=None if act == "none" else Z, act=act, want_dbias=True,
                                      grad_dtype=gd)
        r = ref.backward(A, Bs, [Z], dY, act, gd)
        ref.check(g.dA, r["dA"], "dA %s" % ((M, N, K),))
        ref.check(g.dB, r["dB"][0], "dB %s" % ((M, N, K),))
        ref.check(g.dbias, r["dbias"][0], "dbias %s" % ((M, N, K),))


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_empty_extents(dt):
    d = DT[dt]
    z = lambda m, n: torch.empty((m, n), dtype=d, device="cuda")  # noqa: E731
    gen = torch.Generator().manual_seed(3)
    # no tokens: nothing to write, weight gradients are zero
    assert mk.gated_gemm(z(0, 40), rows(gen, 40, 24, 1, d), rows(gen, 40, 24, 1, d)).shape == (0, 24)
    assert mk.gemm_residual(z(0, 40), rows(gen, 40, 24, 1, d), z(0, 24)).shape == (0, 24)
    g = mk.gated_gemm_backward(z(0, 40), rows(gen, 40, 24, 1, d), rows(gen, 40, 24, 1, d), (z(0, 24), z(0, 24)),
                               z(0, 24), want_dbias=True)
    assert g.dA.shape == (0, 40)
    for t in (g.dBg, g.dBu, g.dbias_g, g.dbias_u):
        assert float(t.abs().sum()) == 0.0
    g = mk.gemm_residual_backward(z(0, 40), rows(gen, 40, 24, 1, d), z(0, 24), want_dbias=True, grad_dtype=d)
    assert float(g.dB.float().abs().sum()) == 0.0 and float(g.dbias.float().abs().sum()) == 0.0
    # no contraction: act of the bias, plus the residual
    b, R = vec(gen, 24, 1.0, d), rows(gen, 5, 24, 1.0, d)
    Y = mk.gemm_residual(z(5, 0), z(0, 24), R, b, act="silu")
    v, e, _ = ref.residual(z(5, 0), z(0, 24), b, R, "silu", d)
    ref.check(Y, (v, e), "K = 0")
    H = mk.gated_gemm(z(5, 0), z(0, 24), z(0, 24), b, b)
    v, e, _, _ = ref.gated(z(5, 0), z(0, 24), z(0, 24), b, b, "silu", d)
    ref.check(H, (v, e), "gated K = 0")
    # no units: the input's gradient is zero
    g = mk.gated_gemm_backward(rows(gen, 5, 40, 1, d), z(40, 0), z(40, 0), (z(5, 0), z(5, 0)), z(5, 0))
    assert float(g.dA.float().abs().sum()) == 0.0


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_unwanted_gradients_and_halves_of_one_weight(dt):
    d = DT[dt]
    M, N, K = 70, 48, 96
    gen, A, _, _ = problem(M, N, K, d)
    W = rows(gen, K, 2 * N, K ** -0.5, d)
    Bg, Bu = W[:, :N], W[:, N:]
    H, Z = mk.gated_gemm_train(A, Bg, Bu)
    assert torch.equal(H, mk.gated_gemm(A, mk.aligned_copy(Bg), mk.aligned_copy(Bu)))
    dY = rows(gen, M, N, 1.0, d)
    full = mk.gated_gemm_backward(A, Bg, Bu, Z, dY, want_dbias=True)
    only = mk.gated_gemm_backward(A, Bg, Bu, Z, dY, want_dB=False)
    assert only.dBg is None and only.dbias_g is None and torch.equal(only.dA, full.dA)
    only = mk.gated_gemm_backward(A, Bg, Bu, Z, dY, want_dA=False)
    assert only.dA is None and torch.equal(only.dBg, full.dBg) and torch.equal(only.dBu, full.dBu)
    dW = torch.zeros((K, 2 * N), dtype=torch.float32, device="cuda")
    mk.gated_gemm_backward(A, Bg, Bu, Z, dY, want_dA=False, dB=(dW[:, :N], dW[:, N:]))
    assert torch.equal(dW[:, :N], full.dBg) and torch.equal(dW[:, N:], full.dBu)


def test_nonfinite_values_stay_in_their_rows():
    # a NaN or infinite token spoils its own row and no other
    d = torch.bfloat16
    _, A, (Bg, Bu), _ = problem(40, 72, 130, d, nb=2)
    clean = mk.gated_gemm(A, Bg, Bu)
    A = A.clone()
    A[3] = float("nan")
    A[17, 5] = float("inf")
    H = mk.gated_gemm(mk.aligned_copy(A), Bg, Bu)
    keep = [i for i in range(40) if i not in (3, 17)]
    assert torch.equal(H[keep], clean[keep]) and bool(torch.isnan(H[3]).all())
    assert not bool(torch.isfinite(H[17]).all())


def test_rows_behind_the_last_stay_as_they_were():
    d = torch.bfloat16
    _, A, (Bg, Bu), _ = problem(19, 40, 64, d, nb=2)
    out = torch.full((32, 48), 3.0, dtype=d, device="cuda")
    mk.gated_gemm(A, Bg, Bu, out=out[:19, :40])
    assert bool((out[19:] == 3.0).all()) and bool((out[:, 40:] == 3.0).all())
