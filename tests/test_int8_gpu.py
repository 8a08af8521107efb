"""The products on 8-bit operands and the quantisation on the GPU: exact integer
sums, 64-bit values within derived bounds, odd extents, padding full of other
bytes, every kernel with the same bits.
"""
import pytest
import torch

import block_reference as ref
import mlp_megakernel_amd as mk
from ffn_reference import U32 as U
from ffn_reference import act_bound
from helpers import progress

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
# single values and tokens, ragged ends of every extent (of K within a pair, a
# 16-byte piece, a slice of 64 and a step of 128 or 256), all few-row forms, small and
# large tiles, contractions that are split
SHAPES = [(1, 1, 1), (1, 5, 3), (1, 100, 16), (2, 17, 64), (3, 33, 65), (16, 64, 127), (17, 40, 128), (31, 129, 129),
          (33, 63, 1001), (48, 16, 255), (64, 250, 257), (65, 257, 130), (100, 72, 4099), (130, 300, 2049),
          (257, 130, 383), (300, 520, 260), (513, 72, 70), (70, 65, 20001), (1, 700, 9999), (640, 1100, 1000)]


def bytes_(gen, rows, cols, pad=0):
    """rows x cols random bytes, -128 among them, in a buffer whose padding holds others."""
    ld = max(16, (cols + 15) // 16 * 16) + 16 * pad
    return torch.randint(-128, 128, (rows, ld), generator=gen, dtype=torch.int8).cuda()[:, :cols]


def scales(gen, n):
    return (torch.rand(n, generator=gen) + 0.5).cuda() / 64


def product(A, B, sa, sb, bias):
    """(value, bound) of z: the sum to fp32, its two scales and the bias, one rounding each."""
    acc = ref.f64(A) @ ref.f64(B).t().contiguous()
    z = acc * (ref.f64(sa)[:, None] * ref.f64(sb)[None, :])
    e = 2.1 * U * z.abs()
    if bias is not None:
        z = z + ref.f64(bias)
    return z, e + U * (z.abs() + e)


def problem(M, N, K, j, nb=1):
    gen = torch.Generator().manual_seed(31 * M + 7 * N + K)
    A, sa = bytes_(gen, M, K, j % 2), scales(gen, M) / max(K, 1) ** 0.5
    Bs, sb = [bytes_(gen, N, K, (j + 1) % 3) for _ in range(nb)], [scales(gen, N) for _ in range(nb)]
    bias = [torch.randn(N, generator=gen).cuda() if j % 3 else None for _ in range(nb)]
    return gen, A, sa, Bs, sb, bias


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("act", ["none", "gelu", "silu", "softplus", "relu"])
def test_plain(out, act):
    od = DT[out]
    for j, (M, N, K) in enumerate(SHAPES):
        progress("int8 %s %s %s" % (out, act, (M, N, K)))
        gen, A, sa, (B,), (sb,), (bias,) = problem(M, N, K, j)
        R = ref.rows(gen, M, N, od, pad=j % 2) if j % 4 else None
        Y, untouched = ref.space(M, N, od, pad=j % 3)
        mk.gemm_int8(A, B, sa, sb, bias, R, act, out=Y)
        z, ez = product(A, B, sa, sb, bias)
        f, ef = act_bound(z, ez, act, False)
        v = f + (ref.f64(R) if R is not None else 0.0)
        ref.check(Y, (v, ref.rounded(v, ef + U * (f.abs() + v.abs()), od)), "Y %s" % ((M, N, K),))
        assert untouched()
        if R is not None:
            R2, untouched = ref.space(M, N, od)
            R2.copy_(R)
            assert torch.equal(mk.gemm_int8(A, B, sa, sb, bias, R2, act, out=R2), Y) and untouched()
        assert torch.equal(mk.gemm_int8(A, B, sa, sb, bias, R, act, out_dtype=od), Y)


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("act", ["silu", "gelu", "none", "relu", "softplus"])
def test_gated(out, act):
    od = DT[out]
    for j, (M, N, K) in enumerate(SHAPES):
        progress("int8 gated %s %s %s" % (out, act, (M, N, K)))
        _, A, sa, Bs, sb, bias = problem(M, N, K, j, 2)
        if j % 2:
            bias[1] = None
        Y, untouched = ref.space(M, N, od, pad=j % 3)
        Bg, Bu = Bs
        mk.gated_gemm_int8(A, Bg, Bu, sa, sb[0], sb[1], bias[0], bias[1], act=act, out=Y)
        (zg, eg), (zu, eu) = product(A, Bg, sa, sb[0], bias[0]), product(A, Bu, sa, sb[1], bias[1])
        f, ef = act_bound(zg, eg, act, False)
        v = f * zu
        e = f.abs() * eu + zu.abs() * ef + ef * eu + U * v.abs()
        ref.check(Y, (v, ref.rounded(v, e, od)), "Y %s" % ((M, N, K),))
        assert untouched()


@pytest.mark.parametrize("gated", [False, True])
def test_a_row_does_not_depend_on_the_others(gated):
    # few rows, small and large tiles, split and whole contractions: one row, one result
    for N, K in ((300, 5000), (1000, 700), (2736, 96)):
        gen, A, sa, Bs, sb, bias = problem(1500, N, K, 1, 2)

        def run(a, b):
            if gated:
                return mk.gated_gemm_int8(A[a:b], *Bs, sa[a:b], *sb, *bias, out_dtype=torch.float32)
            return mk.gemm_int8(A[a:b], Bs[0], sa[a:b], sb[0], bias[0], act="gelu", out_dtype=torch.float32)

        whole = run(0, 1500)
        for a, b in ((0, 1), (5, 8), (20, 40), (100, 150), (200, 264), (300, 400), (500, 900), (1, 1200)):
            progress("rows %d to %d of %s" % (a, b, (N, K)))
            assert torch.equal(run(a, b), whole[a:b])


@pytest.mark.parametrize("M", [1, 20, 50, 200])
def test_the_largest_sums(M):
    K, N = 131071, 24
    A = torch.full((M, 131072), -128, dtype=torch.int8, device="cuda")[:, :K]
    B = torch.full((N, 131072), -128, dtype=torch.int8, device="cuda")[:, :K]
    B[::2] = 127
    one = torch.ones(max(M, N), device="cuda")
    Y = mk.gemm_int8(A, B, one[:M], one[:N], out_dtype=torch.float32)
    want = torch.tensor([-127.0 * 128 * K, 128.0 * 128 * K], dtype=torch.float64).to(torch.float32).repeat(N // 2)
    assert torch.equal(Y.cpu(), want.expand(M, N))


def test_empty_extents_and_no_contraction():
    one = torch.ones(64, device="cuda")
    i8 = lambda m, n: torch.zeros(m, n, dtype=torch.int8, device="cuda")  # noqa: E731
    assert mk.gemm_int8(i8(0, 16), i8(8, 16), one[:0], one[:8]).shape == (0, 8)
    assert mk.gemm_int8(i8(4, 16), i8(0, 16), one[:4], one[:0]).shape == (4, 0)
    for M in (3, 64, 100):
        bias = torch.randn(8, device="cuda")
        s = torch.ones(M, device="cuda")
        Y = mk.gemm_int8(i8(M, 0), i8(8, 0), s, one[:8], bias, act="relu", out_dtype=torch.float32)
        assert torch.equal(Y, bias.clamp(min=0).expand(M, 8))
        H = mk.gated_gemm_int8(i8(M, 0), i8(8, 0), i8(8, 0), s, one[:8], one[:8], bias, bias, act="none",
                               out_dtype=torch.float32)
        assert torch.equal(H, (bias * bias).expand(M, 8))
    q, s = mk.quantize_rows(torch.zeros(5, 0, device="cuda"))
    assert q.shape == (5, 0) and bool((s == 0).all())
    q, s = mk.quantize_columns(torch.zeros(0, 7, device="cuda"))
    assert q.shape == (7, 0) and bool((s == 0).all())
    assert mk.quantize_rows(torch.zeros(0, 8, device="cuda"))[0].shape == (0, 8)


def test_scales_that_are_none():
    # a row without a scale is NaN, the others are as they were
    gen, A, sa, (B,), (sb,), _ = problem(200, 90, 300, 1)
    want = mk.gemm_int8(A, B, sa, sb)
    sa[7], sa[150] = float("nan"), float("inf")
    Y = mk.gemm_int8(A, B, sa, sb)
    good = torch.ones(200, dtype=torch.bool)
    good[[7, 150]] = False
    assert torch.equal(Y[good], want[good]) and bool(Y[7].isnan().all()) and not bool(Y[150].isfinite().any())


# ---------------------------------------------------------------------------
# Quantisation
# ---------------------------------------------------------------------------

def quantized(x):
    """(q, scale) by the definition, each operation in fp32, on the CPU."""
    x = x.float().cpu()
    top = x.abs().amax(1) if x.shape[1] else torch.zeros(x.shape[0])
    full = torch.full_like(top, 127.0)
    q = torch.where(top[:, None] > 0, torch.round(x * (full / top)[:, None]), torch.zeros_like(x))
    return q.to(torch.int8), top / full


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_quantize(dt):
    d = DT[dt]
    for j, (M, N) in enumerate([(1, 1), (5, 3), (3, 8), (9, 65), (4, 511), (7, 513), (2, 1024), (3, 1025), (40, 2731),
                                (2, 4096), (3, 4100), (2, 8193), (1, 16384), (2, 16385), (1, 50001), (130, 200)]):
        progress("quantize %s %s" % (dt, (M, N)))
        gen = torch.Generator().manual_seed(M + N)
        x = ref.rows(gen, M, N, d, std=float(2.0 ** (3 * j - 20 if dt != "f16" else j - 8)), pad=j % 2)
        if M > 3:
            x[2] = 0
        want = quantized(x)
        q, untouched = ref.space(M, (N + 15) // 16 * 16, torch.int8, pad=j % 3, fill=7)
        q.fill_(7)
        got = mk.quantize_rows(x, out=q[:, :N])
        assert torch.equal(got[0].cpu(), want[0]) and torch.equal(got[1].cpu(), want[1])
        assert untouched() and bool((q[:, N:] == 7).all())
        assert int(got[0].min()) >= -127
        # columns: the same of the matrix turned over
        xt = mk.aligned_copy(x.t())
        qc, sc = mk.quantize_columns(xt)
        assert torch.equal(qc, got[0]) and torch.equal(sc, got[1])


def test_quantize_values_that_are_none_and_tiny():
    x = torch.randn(6, 40, device="cuda")
    x[1, 3], x[2, 39], x[3, 0] = float("nan"), float("inf"), float("-inf")
    x[4] *= 1e-42   # subnormal: 127 / amax overflows
    x[5] *= 1e-37
    q, s = mk.quantize_rows(x)
    assert bool((q[1:4] == 0).all()) and bool(s[1:4].isnan().all())
    for r in (0, 4, 5):
        top = x[r].abs().max()
        assert int(q[r][x[r].abs().argmax()].abs()) == 127
        # half a step, and the rounding of scale and quotient
        step = float(top.double()) / 127
        assert float((q[r].double() * step - x[r].double()).abs().max()) <= step * (0.5 + 127 * 4 * U)
    qc, sc = mk.quantize_columns(mk.aligned_copy(x.t()))
    assert torch.equal(qc, q) and torch.equal(sc.nan_to_num(nan=-1.0), s.nan_to_num(nan=-1.0))


def test_a_quantized_layer():
    # weights and tokens quantised, multiplied: within the steps of the two of the exact product
    gen = torch.Generator().manual_seed(4)
    x, W = ref.rows(gen, 100, 500, torch.bfloat16), ref.rows(gen, 500, 300, torch.bfloat16, std=500 ** -0.5)
    (q, s), (qw, sw) = mk.quantize_rows(x), mk.quantize_columns(W)
    Y = mk.gemm_int8(q, qw, s, sw, out_dtype=torch.float32)
    X, V = ref.f64(x), ref.f64(W)
    ex, ev = 0.501 * ref.f64(s)[:, None].expand_as(X), 0.501 * ref.f64(sw)[None, :].expand_as(V)
    e = ex @ V.abs() + X.abs() @ ev + ex @ ev
    ref.check(Y, (X @ V, e * (1 + 1e-6) + 1e-6), "Y")


def test_replays_streams_and_workspaces():
    gen, A, sa, Bs, sb, bias = problem(100, 200, 9000, 1, 2)
    x = ref.rows(gen, 100, 9000, torch.bfloat16)
    R = ref.rows(gen, 100, 200, torch.bfloat16)

    def step():
        q, s = mk.quantize_rows(x)
        return (q, s, mk.gemm_int8(q, Bs[0], s, sb[0], bias[0], R, "gelu"),
                mk.gated_gemm_int8(q[:9], *Bs, s[:9], *sb, *bias))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        held = step()
    for _ in range(4):
        x.mul_(1.25)
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))
    torch.cuda.synchronize()
    q, s = mk.quantize_rows(x, stream=side)
    y = mk.gemm_int8(q, Bs[0], s, sb[0], bias[0], R, "gelu", stream=side)
    z = mk.gated_gemm_int8(q, *Bs, s, *sb, *bias, stream=side)
    side.synchronize()
    assert torch.equal(q, want[0]) and torch.equal(y, want[2]) and torch.equal(z[:9], want[3])


def test_far_rows():
    # operands above 2 GiB: the last rows as by themselves
    M, K = 70000, 32784
    A = torch.randint(-128, 128, (M, K), dtype=torch.int8, device="cuda")
    B, s = torch.randint(-128, 128, (40, K), dtype=torch.int8, device="cuda"), torch.ones(M, device="cuda")
    Y = mk.gemm_int8(A, B, s, s[:40], out_dtype=torch.float32)
    assert torch.equal(Y[-5:], mk.gemm_int8(A[-5:], B, s[:5], s[:40], out_dtype=torch.float32))
    Z = mk.gemm_int8(B[:3], A, s[:3], s, out_dtype=torch.float32)
    assert torch.equal(Z, Y.t()[:3])


def test_refusals():
    A = torch.zeros(4, 32, dtype=torch.int8, device="cuda")
    s = torch.ones(4, device="cuda")
    x = torch.zeros(4, 32, device="cuda")
    for c in (lambda: mk.gemm_int8(x, A, s, s), lambda: mk.gemm_int8(A, x, s, s), lambda: mk.gemm_int8(A, A, s[:3], s),
              lambda: mk.gemm_int8(A, A, s.half(), s), lambda: mk.gemm_int8(A, A[:, :16], s, s),
              lambda: mk.gemm_int8(A, A, s, s, s.half()), lambda: mk.gemm_int8(A, A, s, s, act="tanh"),
              lambda: mk.gemm_int8(A, A, s, s, out_dtype=torch.int32), lambda: mk.gemm_int8(A, A.cpu(), s, s),
              lambda: mk.gemm_int8(A, A, s, s, residual=x), lambda: mk.gated_gemm_int8(A, A, A[:3], s, s, s),
              lambda: mk.gated_gemm_int8(A, A, A, s, s, s[:2]), lambda: mk.quantize_rows(A),
              lambda: mk.quantize_rows(x[0]),
              lambda: mk.quantize_rows(x, out=A[:2]), lambda: mk.quantize_columns(x, out=A),
              lambda: mk.quantize_rows(x, scale=s[:2])):
        with pytest.raises(ValueError):
            c()
    B = torch.zeros(4, 40, dtype=torch.int8, device="cuda")
    for c in (lambda: mk.gemm_int8(B, B, s, s), lambda: mk.gemm_int8(A[:, 1:], A[:, 1:], s, s),
              lambda: mk.quantize_rows(torch.zeros(4, 33, device="cuda"))):
        with pytest.raises(mk.CoalesceError):
            c()
