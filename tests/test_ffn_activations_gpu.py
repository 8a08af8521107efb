"""The activations of the feed-forward operators where their values are small or
not finite, on every kernel that applies them: the few-row kernel, whole and
ragged tiles, and the pass that joins a split contraction.

The pre-activations are exact: each output column n picks the contraction index
n mod 16 with a weight of one, so z[m][n] = A[m][n mod 16] and every other
product is zero.  What is left is the activation's own error, a product or a sum
in fp32 (half a step, 2^-24) and the rounding of the result."""
import pytest
import torch

import ffn_reference as ref
import mlp_megakernel_amd as mk
from helpers import progress

pytestmark = pytest.mark.gpu

# rows, columns, contraction: few rows in strips of 16, 32 and 64; whole and
# ragged tiles of every height; split contractions
SHAPES = [(1, 40, 64), (17, 4100, 64), (40, 8200, 72), (64, 200, 64), (65, 40, 64), (70, 300, 4100), (500, 1030, 4100),
          (1300, 1030, 64), (3000, 1030, 64), (4100, 5461, 130), (8192, 4096, 64)]
# Relative errors in units of 2^-24; the hardware's exponential, logarithm and
# reciprocal are good to 1 ulp (2 units).
#  * gelu: nine Horner steps of positive terms (1 unit each) with coefficients
#    rounded to fp32 (1 each for numerator and denominator), reciprocal 2,
#    exponential 2, three products 3: 18; the exponent z^2 (-log2(e) / 2) carries
#    2.5 roundings, z^2 / 2 times 2.5 units in the exponential: 1.25 z^2.  The fit
#    itself is good to 5.1e-9 (0.1 units).
def gelu_rel(z):
    return (18.5 + 1.25 * z * z) * ref.U32


def pick(M, N, K, dt, values):
    """A, B with A @ B = the values, in turn over rows and the first 16 indices of the contraction."""
    n = M * 16
    A = torch.zeros(M, (K + 7) // 8 * 8, dtype=dt, device="cuda")
    A[:, :16] = values.to(dt).repeat((n + values.numel() - 1) // values.numel())[:n].view(M, 16)
    B = torch.zeros(K, (N + 7) // 8 * 8, dtype=dt, device="cuda")
    c = torch.arange(N, device="cuda")
    B[c % 16, c] = 1.0
    z = A[:, :16].double()[:, c.remainder(16)]
    return A[:, :K], B[:, :N], z


FLUSH = 2.0 ** -126     # what is below may be taken as zero


def within(got, v, e, dtype, what):
    ref.check(got, (v, ref.rounded(v, e, dtype) + FLUSH), what)


def gelu64(z):
    return z * 0.5 * torch.erfc(-z / 2.0 ** 0.5)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("out32", [False, True])
def test_gelu_keeps_its_tail(dt, out32):
    od = torch.float32 if out32 else dt
    # the tail, both sides of zero, and far beyond
    zs = torch.cat([torch.linspace(-14.0, 9.0, 1187), torch.tensor([-1000.0, -100.0, -20.0, 0.0, 1e-4, -1e-4, 20.0])])
    for shape in SHAPES:
        M, N, K = shape
        A, B, z = pick(M, N, K, dt, zs.cuda())
        up = 64.0
        f = gelu64(z)
        e = f.abs() * gelu_rel(z) + z.abs() * FLUSH    # the exponential flushed
        Y = mk.gemm_residual(A, B, act="gelu", out_dtype=od)
        within(Y, f, e, od, "act %s" % (shape,))
        # times u = 64 z
        H = mk.gated_gemm(A, B, mk.aligned_copy(B * up), act="gelu", out_dtype=od)
        v = f * (up * z)
        within(H, v, (up * z).abs() * e + ref.U32 * v.abs(), od, "gated %s" % (shape,))
        progress("gelu %s %s %s" % (dt, od, shape))


def grads(zs, dt, act):
    """act(z) and act'(z) in fp32 as the backward takes them: the bias gradients of one row, dY = Zu = 1."""
    n = zs.numel()
    z = zs.to(dt).cuda()[None, :].contiguous()
    one = torch.ones_like(z)
    A, B = torch.zeros(1, 8, dtype=dt, device="cuda"), torch.zeros(8, n, dtype=dt, device="cuda")
    g = mk.gated_gemm_backward(A, B, B, (z, one), one.float(), act=act, want_dA=False, want_dB=False, want_dbias=True)
    r = mk.gemm_residual_backward(A, B, one, z, act=act, want_dA=False, want_dB=False, want_dbias=True)
    assert torch.equal(r.dbias, g.dbias_g)
    return z[0].double(), g.dbias_u, g.dbias_g


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_gelu_of_the_backward(dt):
    zs = torch.cat([torch.linspace(-14.0, 9.0, 4094), torch.tensor([-1000.0, 0.0])])
    z, f, d = grads(zs, dt, "gelu")
    v, u = gelu64(z), ref.U32
    ref.check(f, (v, v.abs() * gelu_rel(z) + z.abs() * FLUSH + FLUSH), "gelu")
    # Phi(z) + z phi(z): the two terms' errors (phi: exponential 2, constant and
    # two products 3) and the sum's rounding
    cdf, zphi = 0.5 * torch.erfc(-z / 2.0 ** 0.5), z * torch.exp(-z * z / 2) / (2 * torch.pi) ** 0.5
    e = cdf * gelu_rel(z) + zphi.abs() * (5 + 1.25 * z * z) * u + (cdf + zphi).abs() * u
    ref.check(d, (cdf + zphi, e + z.abs() * FLUSH + FLUSH), "gelu'")


# Hardware exponential of z log2(e) (constant and product rounded: 1.5 |z| units,
# its own ulp 2), as the sigmoid adds 1 (1 unit) and takes a reciprocal (2).
def sigmoid_rel(z):
    return (5 + 1.5 * z.abs()) * ref.U32


def softplus64(z):
    return torch.clamp(z, min=0) + torch.log1p(torch.exp(-z.abs()))


def softplus_err(z):
    """Below ln(2^-5) the series of ln(1 + t): t's error, two products, 0.1 for the terms left out.  Above, 1 + t is
    rounded (1 unit of 1 + t, so of the logarithm) with t's error beside it, then the logarithm (2) and its base
    change (1.5).  Above 20 z itself: e^-20 is below a unit."""
    u, f, t = ref.U32, softplus64(z), torch.exp(torch.clamp(z, max=20.0))
    et = (2 + 1.5 * z.abs()) * u
    return torch.where(z < -3.4, f * (et + 2.1 * u), torch.zeros_like(f)) + \
        torch.where((z > -3.5) & (z <= 20), u + et * t / (1 + t) + 3.5 * u * f, u * f.abs()) + FLUSH


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("out32", [False, True])
def test_softplus_keeps_its_tail(dt, out32):
    od = torch.float32 if out32 else dt
    zs = torch.cat([torch.linspace(-40.0, 25.0, 1187), torch.tensor([-100.0, -17.5, -10.0, 0.0, 1e-4])])
    for shape in SHAPES:
        A, B, z = pick(*shape, dt, zs.cuda())
        f, e = softplus64(z), softplus_err(z)
        within(mk.gemm_residual(A, B, act="softplus", out_dtype=od), f, e, od, "act %s" % (shape,))
        H = mk.gated_gemm(A, B, mk.aligned_copy(B * 32.0), act="softplus", out_dtype=od)
        v = f * (32.0 * z)
        within(H, v, (32.0 * z).abs() * e + ref.U32 * v.abs(), od, "gated %s" % (shape,))
        progress("softplus %s %s %s" % (dt, od, shape))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_softplus_of_the_backward(dt):
    z, f, d = grads(torch.cat([torch.linspace(-40.0, 25.0, 4093), torch.tensor([-100.0, -17.5, 0.0])]), dt, "softplus")
    ref.check(f, (softplus64(z), softplus_err(z)), "softplus")
    s = torch.sigmoid(z)
    ref.check(d, (s, s * sigmoid_rel(z) + 2 * FLUSH), "softplus'")


# The formulas at values that are not finite, as 64-bit arithmetic evaluates
# them: z Phi(z) and z sigma(z) at minus infinity are -inf * 0.
NAN, INF = float("nan"), float("inf")
NONFINITE = {"none": (NAN, INF, -INF), "relu": (NAN, INF, 0.0), "silu": (NAN, INF, NAN), "gelu": (NAN, INF, NAN),
             "softplus": (NAN, INF, 0.0)}


@pytest.mark.parametrize("act", sorted(NONFINITE))
@pytest.mark.parametrize("out32", [False, True])
def test_values_that_are_not_finite(act, out32):
    d = torch.bfloat16
    od = torch.float32 if out32 else d
    want = torch.tensor(NONFINITE[act], device="cuda", dtype=torch.float64)
    for M, N, K in SHAPES:
        # z[m][n] = A[m][0]: rows of NaN, infinity, minus infinity and 1.5 in turn
        A = torch.zeros(M, (K + 7) // 8 * 8, dtype=d, device="cuda")
        A[:, 0] = torch.tensor([NAN, INF, -INF, 1.5], device="cuda").repeat((M + 3) // 4)[:M]
        B = torch.zeros(K, (N + 7) // 8 * 8, dtype=d, device="cuda")
        B[0] = 1.0
        A, B = A[:, :K], B[:, :N]
        R = torch.full((M, (N + 7) // 8 * 8), 2.0, dtype=od, device="cuda")[:, :N]
        Y = mk.gemm_residual(A, B, R, act=act, out_dtype=od)
        H = mk.gated_gemm(A, B, B, act=act, out_dtype=od)
        for i in range(min(M, 3)):
            y = torch.full_like(Y[i::4], float(want[i] + 2.0))
            h = torch.full_like(H[i::4], float(want[i] * (NAN, INF, -INF)[i]))
            assert torch.equal(Y[i::4].nan_to_num(nan=7.0), y.nan_to_num(nan=7.0)), (act, M, N, K, i)
            assert torch.equal(H[i::4].nan_to_num(nan=7.0), h.nan_to_num(nan=7.0)), (act, M, N, K, i)
        assert bool(torch.isfinite(Y[3::4]).all()) and bool(torch.isfinite(H[3::4]).all())


def test_relu_of_the_backward_keeps_nan():
    z, f, d = grads(torch.tensor([NAN, -1.0, 0.0, 2.0]), torch.bfloat16, "relu")
    assert bool(torch.isnan(f[0])) and f[1:].tolist() == [0.0, 0.0, 2.0] and d.tolist() == [0.0, 0.0, 0.0, 1.0]
