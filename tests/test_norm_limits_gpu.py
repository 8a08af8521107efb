"""Layer norm and its gradients at the edges of their range: rows whose values, mean or
deviations are far from 1, against 64-bit references."""
import numpy as np
import pytest
import torch

import block_reference as ref
import mlp_megakernel_amd as mk
from ffn_reference import U32 as U
from helpers import progress

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f32"), ("f32", "f32")]
# each form of the kernels, with columns of the last thread outside the row, and one that its row fills
WIDTHS = [100, 701, 1500, 2048, 3001, 5000, 9003, 16400]


def check_backward(S, w, stats, dy, dsum, mask, dt, what, branch=True):
    g = mk.layer_norm_backward(S, w, stats, dy, dsum, *mask, want_dbranch=branch)
    r = ref.norm_backward(S, w, *stats, dy, dsum, mask, dt, S.dtype, torch.float32)
    for name in ("dx", "dbranch", "dweight", "dbias") if branch else ("dx", "dweight", "dbias"):
        ref.check(getattr(g, name), r[name], "%s of %s" % (name, what))


@pytest.mark.parametrize("types", TYPES, ids="-".join)
@pytest.mark.parametrize("p", [0.0, 0.25])
def test_backward_of_far_rows_without_deviation(types, p):
    # |mean| rstd is beyond fp32 in rows 1 and 3, but xh = (s - mean) rstd is 0 everywhere in them.  Their rstd
    # is 2^33.2, and the weights take that out of their gradients (which fp16 would not hold).
    dt, sdt = DT[types[0]], DT[types[1]]
    for N in WIDTHS:
        progress("far rows %s %s %d" % (types, p, N))
        gen = torch.Generator().manual_seed(N)
        S = ref.rows(gen, 5, N, sdt)
        S[1], S[3] = 2.0 ** 100, -2.0 ** 100
        w = (2.0 ** -33 * torch.randn(N, generator=gen)).cuda()
        dy, dsum = ref.rows(gen, 5, N, dt), ref.rows(gen, 5, N, sdt)
        _, stats = mk.layer_norm_train(S, w, eps=1e-20, out_dtype=dt)
        assert bool((stats[0][[1, 3]].abs() == 2.0 ** 100).all()) and bool((stats[1][[1, 3]] > 2.0 ** 33).all())
        for ds in (dsum, None):
            check_backward(S, w, stats, dy, ds, (p, 7, 1), dt, N)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_backward_of_a_constant_row(dt):
    # at the default eps
    gen = torch.Generator().manual_seed(1)
    S = ref.rows(gen, 1, 100, DT[dt])
    S.fill_(2.0 ** 120)
    y, stats = mk.layer_norm_train(S)
    assert bool((y == 0).all())
    check_backward(S, None, stats, ref.rows(gen, 1, 100, DT[dt]), None, (0.0, 0, 0), DT[dt], "a constant row")


# ---------------------------------------------------------------------------
# Forward
# ---------------------------------------------------------------------------

def norm64(s, w, b, eps, dt):
    """dict of (value, bound) of y, mean and rstd of a stream s, whose mean is corrected where it is large.

    The mean found first is off by at most DEPTH + 1 roundings of the values' mean size; the deviations d from it
    are off by one rounding each.  Where its square is above the variance and eps (half as much again, so that
    this and the kernel's own values agree), the mean of d is found by so many roundings of the size of d and
    taken from them, which leaves a second-order term of the first error.
    """
    s = ref.f64(s)
    eps = float(np.float32(eps))
    k = min(s.shape[1], ref.DEPTH) + 2
    mean = s.mean(1, keepdim=True)
    dev = s - mean
    var = dev.square().mean(1, keepdim=True)
    e0 = k * U * s.abs().mean(1, keepdim=True)
    size = dev.abs() + e0                                 # of d
    em = torch.where(mean.square() > 1.5 * (var + eps), k * U * size.mean(1, keepdim=True), e0)
    ed = em + 3 * U * size                                # d's rounding, that of its mean and of their difference
    ev = (2 * dev.abs() * ed + ed * ed).mean(1, keepdim=True)
    ev = ev + (k + 3) * U * (var + ev)
    rstd = 1 / torch.sqrt(var + eps)
    hi, lo = 1 / torch.sqrt(torch.clamp(var - ev, min=0) + eps), 1 / torch.sqrt(var + ev + eps)
    er = torch.maximum(hi - rstd, rstd - lo) + 3 * U * hi
    t = dev * rstd
    et = ed * rstd + dev.abs() * er + ed * er + U * (t.abs() + ed * hi)
    y = t * ref.f64(w) + ref.f64(b)
    ey = et * ref.f64(w).abs() + U * (y.abs() + et * ref.f64(w).abs())
    return {"y": (y, ref.rounded(y, ey, dt)), "mean": (mean[:, 0], (em + U * (mean.abs() + em))[:, 0]),
            "rstd": (rstd[:, 0], er[:, 0])}


def check_forward(S, w, b, eps, dt, what):
    y, (mean, rstd) = mk.layer_norm_train(S, w, b, eps=eps, out_dtype=dt)
    r = norm64(S, w, b, eps, dt)
    for got, name in ((y, "y"), (mean, "mean"), (rstd, "rstd")):
        ref.check(got, r[name], "%s of %s" % (name, what))
    return y, mean, rstd


def affine(N, seed):
    gen = torch.Generator().manual_seed(seed)
    return gen, (1 + 0.3 * torch.randn(N, generator=gen)).cuda(), (0.3 * torch.randn(N, generator=gen)).cuda()


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_rows_far_from_zero(dt):
    # constant rows whose sums are not exact: y is the bias; and rows of unit deviation, or of some steps of
    # their own type, around a far mean
    for N in WIDTHS + [96, 768, 1000, 4096, 16384, 40001]:
        progress("far from zero %s %d" % (dt, N))
        gen, w, b = affine(N, N)
        S = ref.rows(gen, 9, N, torch.float32)
        S[0], S[1], S[2], S[3] = 1000.1, 12345.678, 100000.3, -3.1e7
        S[4:] += torch.tensor([1000.1, 12345.678, -100000.3, 4096.0, 1e6], device="cuda")[:, None]
        check_forward(S, w, b, 1e-5, DT[dt], N)
        # the same as the sum of a stream and a branch (exact: the halves of each value)
        half = ref.rows(gen, 9, N, torch.float32)
        half.copy_(S * 0.5)
        if dt == "f32":
            y, s, _ = mk.add_layer_norm_train(half, half, w, b)
            assert torch.equal(s, S) and torch.equal(y, mk.layer_norm(S, w, b))


@pytest.mark.parametrize("types", TYPES, ids="-".join)
def test_deviations_whose_squares_leave_fp32(types):
    # 2^70 and 2^100 overflow when squared, 2^-70 and 2^-100 vanish, and without an eps they count
    dt, sdt = DT[types[0]], DT[types[1]]
    for N in WIDTHS + [4096]:
        progress("range %s %d" % (types, N))
        gen, w, b = affine(N, N)
        S = ref.rows(gen, 7, N, sdt, mean=0.25)
        S *= torch.tensor([2.0 ** k for k in (70, 100, -70, -100, 0, -45, 60)], device="cuda", dtype=sdt)[:, None]
        y, mean, rstd = check_forward(S, w, b, 0.0, dt, N)
        dy = ref.rows(gen, 7, N, dt)
        check_backward(S, w, (mean, rstd), dy, None, (0.0, 0, 0), dt, N, branch=dt is not torch.float16)
        # beside an eps the small ones are nothing, and the large ones as before
        again, _, _ = check_forward(S, w, b, 1e-5, dt, N)
        assert torch.equal(again[[0, 1, 6]], y[[0, 1, 6]])


@pytest.mark.parametrize("given", [False, True])
def test_statistics_of_rows_without_columns(given):
    # 0 / 0, whatever the memory held
    x = torch.empty(5, 0, device="cuda", dtype=torch.bfloat16)
    for stream in (None, torch.cuda.Stream()):
        for call in (lambda **kw: mk.layer_norm_train(x, stream=stream, **kw),
                     lambda **kw: mk.add_layer_norm_train(x, x, stream=stream, **kw)):
            torch.full((1 << 12,), 3.0, device="cuda")  # (freed: what comes next may hold it)
            stats = tuple(torch.full((5,), 7.0, device="cuda") for _ in range(2)) if given else None
            torch.cuda.synchronize()
            got = call(stats=stats)
            torch.cuda.synchronize()
            assert got[0].shape == (5, 0)
            for i in range(2):
                assert got[-1][i].shape == (5,) and bool(got[-1][i].isnan().all())
                assert not given or got[-1][i] is stats[i]
            _, (mean, rstd) = mk.layer_norm_train(x, stats=(got[-1][0].zero_(), None))  # one of them
            assert bool(mean.isnan().all()) and rstd is None
