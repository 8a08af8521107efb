"""GPU parity of layer norm, its fused form and its gradients with 64-bit
references, within bounds derived per element (block_reference.py): odd extents,
padded pitches, every type, rows of one value and longer than the registers,
in-place sums, masked-out NaN, neighbours left as they were.
"""
import pytest
import torch

import block_reference as ref
import mlp_megakernel_amd as mk
from helpers import progress

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32"), ("f32", "f32")]
# every form of the kernels: one wave per row (up to 1024), one workgroup (up to
# 16384), passes over longer ones; and the edges between them
SHAPES = [(1, 1), (3, 2), (2, 7), (5, 8), (9, 65), (4, 511), (7, 512), (3, 513), (6, 1001), (5, 1024), (2, 1025),
          (3, 2048), (2, 2731), (1, 4096), (3, 4097), (2, 8192), (2, 8195), (1, 16384), (2, 16385), (1, 40001)]


def setup(M, N, dt, sdt, j, seed=0):
    gen = torch.Generator().manual_seed(seed + 7919 * M + N)
    wt = torch.float32 if j % 3 == 2 else dt
    w = (1 + 0.3 * torch.randn(N, generator=gen)).to(wt).cuda() if j % 4 != 3 else None
    b = (0.3 * torch.randn(N, generator=gen)).to(wt).cuda() if j % 4 < 2 else None
    S = ref.rows(gen, M, N, sdt, mean=0.7, std=1.5, pad=j % 2)
    X = ref.rows(gen, M, N, dt, pad=(j + 1) % 2)
    return gen, w, b, S, X


@pytest.mark.parametrize("types", TYPES, ids="-".join)
def test_norm(types):
    dt, sdt = DT[types[0]], DT[types[1]]
    for j, (M, N) in enumerate(SHAPES):
        progress("norm %s %s" % (types, (M, N)))
        _, w, b, S, _ = setup(M, N, dt, sdt, j)
        r = ref.norm(S, None, w, b, 1e-5, None, dt, sdt)
        out, untouched = ref.space(M, N, dt, pad=j % 3)
        y, (mean, rstd) = mk.layer_norm_train(S, w, b, out=out)
        ref.check(y, r["y"], "y %s" % ((M, N),))
        ref.check(mean, r["mean"], "mean %s" % ((M, N),))
        ref.check(rstd, r["rstd"], "rstd %s" % ((M, N),))
        assert y is out and untouched()
        assert torch.equal(mk.layer_norm(S, w, b, out_dtype=dt), y)


@pytest.mark.parametrize("types", TYPES, ids="-".join)
@pytest.mark.parametrize("p", [0.0, 0.1, 0.75])
def test_norm_of_a_sum(types, p):
    dt, sdt = DT[types[0]], DT[types[1]]
    for j, (M, N) in enumerate(SHAPES):
        progress("sum %s %s %s" % (types, p, (M, N)))
        _, w, b, S, X = setup(M, N, dt, sdt, j, 1)
        seed, offset = 0x123456789ABCDEF + j, (j << 33) + 5
        r = ref.norm(X, S, w, b, 1e-6, (p, seed, offset), dt, sdt)
        sum_out, untouched = ref.space(M, N, sdt, pad=j % 3)
        y, s, (mean, rstd) = mk.add_layer_norm_train(X, S, w, b, eps=1e-6, p=p, seed=seed, offset=offset,
                                                     sum_out=sum_out)
        for got, name in ((y, "y"), (s, "sum"), (mean, "mean"), (rstd, "rstd")):
            ref.check(got, r[name], "%s %s" % (name, (M, N)))
        assert untouched()
        # in place, from a seed in device memory, without statistics: the same bits
        R2, untouched = ref.space(M, N, sdt)
        R2.copy_(S)
        both = torch.tensor([seed, offset], device="cuda")
        y2, s2 = mk.add_layer_norm(X, R2, w, b, eps=1e-6, p=p, seed=both, sum_out=R2)
        assert torch.equal(y2, y) and torch.equal(s2, s) and s2 is R2 and untouched()


@pytest.mark.parametrize("types", TYPES, ids="-".join)
@pytest.mark.parametrize("p", [0.0, 0.25])
def test_norm_backward(types, p):
    dt, sdt = DT[types[0]], DT[types[1]]
    for j, (M, N) in enumerate(SHAPES + [(700, 40), (1100, 520), (1030, 1500), (9, 16400)]):
        progress("backward %s %s %s" % (types, p, (M, N)))
        gen, w, _, S, _ = setup(M, N, dt, sdt, j, 2)
        dy = ref.rows(gen, M, N, dt, pad=j % 2)
        dsum = ref.rows(gen, M, N, sdt, pad=1) if j % 3 else None
        _, (mean, rstd) = mk.layer_norm_train(S, w, out_dtype=dt)
        gd = dt if j % 2 else torch.float32
        mask = (p, 99 + j, 3)
        dx, ux = ref.space(M, N, sdt, pad=j % 3)
        db, ub = ref.space(M, N, dt, pad=j % 2)
        g = mk.layer_norm_backward(S, w, (mean, rstd), dy, dsum, *mask, want_dbranch=True, grad_dtype=gd, dx=dx,
                                   dbranch=db)
        r = ref.norm_backward(S, w, mean, rstd, dy, dsum, mask, dt, sdt, gd)
        for name in ("dx", "dbranch", "dweight", "dbias"):
            ref.check(getattr(g, name), r[name], "%s %s" % (name, (M, N)))
        assert ux() and ub()
        # each by itself, and the stream's gradient formed in place: the same bits
        g1 = mk.layer_norm_backward(S, w, (mean, rstd), dy, dsum, want_dweight=False, want_dbias=False)
        g2 = mk.layer_norm_backward(S, w, (mean, rstd), dy, want_dx=False, want_dweight=False, grad_dtype=gd)
        assert torch.equal(g1.dx, g.dx) and torch.equal(g2.dbias, g.dbias)
        assert g1.dweight is g1.dbias is g2.dx is g2.dweight is None
        if dsum is not None:
            acc, uacc = ref.space(M, N, sdt)
            acc.copy_(dsum)
            g3 = mk.layer_norm_backward(S, w, (mean, rstd), dy, acc, dx=acc, want_dweight=False, want_dbias=False)
            assert torch.equal(g3.dx, g.dx) and uacc()


def test_gradient_against_differences():
    # d(sum c y) along a direction, in steps of 2^-8 of fp32 inputs of unit size:
    # truncation h^2 |f'''| / 6 and the rounding of y, 2^-22 sqrt(M N) / h, both
    # below 1e-3 of the derivative's scale sqrt(M N)
    gen = torch.Generator().manual_seed(5)
    M, N, h = 6, 200, 2.0 ** -8
    S, w = ref.rows(gen, M, N, torch.float32), (1 + 0.2 * torch.randn(N, generator=gen)).cuda()
    c, v = (torch.randn(M, N, generator=gen).cuda() for _ in range(2))
    y, st = mk.layer_norm_train(S, w)
    g = mk.layer_norm_backward(S, w, st, c)

    def f(s, w):
        return float((f64(mk.layer_norm(s, w)) * f64(c)).sum())

    f64 = ref.f64
    for got, plus, minus in (
            (float((f64(g.dx) * f64(v)).sum()), f(mk.aligned_copy(S + h * v), w), f(mk.aligned_copy(S - h * v), w)),
            (float((f64(g.dweight) * f64(v[0])).sum()), f(S, w + h * v[0]), f(S, w - h * v[0]))):
        assert abs((plus - minus) / (2 * h) - got) <= 1e-3 * (M * N) ** 0.5


@pytest.mark.parametrize("N", [40, 700, 2731, 16500])
def test_values_that_are_none(N):
    # a NaN or an infinity makes its own row NaN and no other; so with the gradients
    gen = torch.Generator().manual_seed(N)
    S = ref.rows(gen, 9, N, torch.bfloat16)
    clean, st0 = mk.layer_norm_train(S)
    dy = ref.rows(gen, 9, N, torch.bfloat16)
    g0 = mk.layer_norm_backward(S, None, st0, dy, want_dweight=False, want_dbias=False)
    T = S.clone() if S.is_contiguous() else mk.aligned_copy(S)
    T[2, N // 2], T[5, 0], T[7, N - 1] = float("nan"), float("inf"), float("-inf")
    y, st = mk.layer_norm_train(T)
    g = mk.layer_norm_backward(T, None, st, dy, want_dweight=False, want_dbias=False)
    bad = torch.zeros(9, dtype=torch.bool)
    bad[[2, 5, 7]] = True
    assert bool(y[bad].isnan().all()) and torch.equal(y[~bad], clean[~bad])
    assert bool(g.dx[bad].isnan().all()) and torch.equal(g.dx[~bad], g0.dx[~bad])


@pytest.mark.parametrize("N", [1, 96, 1024, 5000])
def test_constant_rows_and_large_means(N):
    # no deviation: y is the bias; a mean of 2^12 with unit deviations keeps them
    gen = torch.Generator().manual_seed(N)
    w, b = torch.randn(N, generator=gen).cuda(), torch.randn(N, generator=gen).cuda()
    S = mk.aligned_empty(4, N, torch.float32)
    S.copy_(torch.tensor([0.0, 3.0, -2.0 ** 20, 2.0 ** -100])[:, None].expand(4, N))
    assert torch.equal(mk.layer_norm(S, w, b), b[None, :].expand(4, N))
    T = ref.rows(gen, 5, N, torch.float32, mean=4096.0)
    y, (mean, rstd) = mk.layer_norm_train(T, w, b)
    r = ref.norm(T, None, w, b, 1e-5, None, torch.float32, torch.float32)
    ref.check(y, r["y"], "y")
    ref.check(rstd, r["rstd"], "rstd")


def test_empty_extents():
    for M, N in ((0, 40), (5, 0), (0, 0)):
        x = torch.empty(M, N, device="cuda", dtype=torch.bfloat16)
        st = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
        assert mk.layer_norm(x).shape == (M, N)
        g = mk.layer_norm_backward(x, None, st, x, want_dbranch=True)
        assert g.dx.shape == g.dbranch.shape == (M, N) and g.dweight.shape == (N,)
        assert bool((g.dweight == 0).all()) and bool((g.dbias == 0).all())


def test_halves_of_one_matrix():
    # the operands of one pitch lie between each other's rows
    gen = torch.Generator().manual_seed(3)
    both = ref.rows(gen, 30, 2 * 104, torch.bfloat16)
    x, out = both[:, :101], both[:, 104:205]
    want = mk.layer_norm(mk.aligned_copy(x))
    rest = both[:, 101:104].clone(), both[:, 205:].clone()
    assert torch.equal(mk.layer_norm(x, out=out), want)
    assert torch.equal(both[:, 101:104], rest[0]) and torch.equal(both[:, 205:], rest[1])


def test_far_rows():
    # element offsets beyond 2^31: the last rows of a tall matrix equal the same rows by themselves
    M, N = (1 << 21) + 5, 1030
    S = torch.empty(M, 1032, device="cuda", dtype=torch.bfloat16)[:, :N]
    S.normal_(0.5, 1.0, generator=torch.Generator(device="cuda").manual_seed(1))
    y, st = mk.layer_norm_train(S)
    assert torch.equal(y[-7:], mk.layer_norm(S[-7:]))
    g = mk.layer_norm_backward(S, None, st, y, want_dweight=False, want_dbias=False)
    tail = mk.layer_norm_backward(S[-7:], None, tuple(t[-7:].clone() for t in st), y[-7:], want_dweight=False,
                                  want_dbias=False)
    assert torch.equal(g.dx[-7:], tail.dx)


def test_replays_and_streams():
    gen = torch.Generator().manual_seed(11)
    M, N = 300, 1500
    S, X, dy = (ref.rows(gen, M, N, torch.bfloat16) for _ in range(3))
    w = (1 + 0.1 * torch.randn(N, generator=gen)).bfloat16().cuda()
    both = torch.tensor([7, 0], device="cuda")

    def step():
        y, s, st = mk.add_layer_norm_train(X, S, w, p=0.2, seed=both)
        g = mk.layer_norm_backward(s, w, st, dy, y, 0.2, both, want_dbranch=True)
        return (y, s, *st, *g)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        held = step()
    masks = []
    for i in range(4):
        both.copy_(torch.tensor([7 + i // 2, i]))
        S.add_(0.25)
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, want):
            assert torch.equal(a, b)
        masks.append(held[-3] == 0)
    assert all(not torch.equal(masks[0], m) for m in masks[1:])
    want = step()
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_binding_refuses():
    x = torch.zeros(4, 32, device="cuda", dtype=torch.bfloat16)
    f, v = x.float(), torch.zeros(32, device="cuda")
    st = torch.zeros(4, device="cuda"), torch.ones(4, device="cuda")
    calls = [lambda: mk.layer_norm(x.long()), lambda: mk.layer_norm(x[0]), lambda: mk.layer_norm(x.t()),
             lambda: mk.layer_norm(x.cpu()), lambda: mk.layer_norm(x, out_dtype=torch.float32),
             lambda: mk.layer_norm(x, v[:16]), lambda: mk.layer_norm(x, v.half()),
             lambda: mk.layer_norm(x, v, v.bfloat16()),
             lambda: mk.layer_norm(x, out=x[:2].clone()), lambda: mk.add_layer_norm(x, f[:2]),
             lambda: mk.add_layer_norm(x, x.half()), lambda: mk.add_layer_norm(f, x),
             lambda: mk.add_layer_norm(x, x, seed=torch.zeros(1, device="cuda", dtype=torch.int64)),
             lambda: mk.add_layer_norm(x, x, seed=torch.zeros(2, dtype=torch.int64)),
             lambda: mk.add_layer_norm(x, x, seed=torch.zeros(2, device="cuda", dtype=torch.int64), offset=1),
             lambda: mk.layer_norm_backward(x, None, st[:1], x), lambda: mk.layer_norm_backward(x, None, st, f),
             lambda: mk.layer_norm_backward(x, None, (st[0][:2], st[1]), x),
             lambda: mk.layer_norm_backward(f, None, st, x, dsum=x),
             lambda: mk.layer_norm_backward(x, None, st, x, grad_dtype=torch.float16)]
    for i, c in enumerate(calls):
        with pytest.raises(ValueError):
            c()
            raise AssertionError("call %d was accepted" % i)
    for c in (lambda: mk.layer_norm(x, out=x), lambda: mk.add_layer_norm(x, x, p=1.5),
              lambda: mk.layer_norm(x, eps=-1.0), lambda: mk.layer_norm(x, eps=float("nan")),
              lambda: mk.layer_norm(torch.zeros(4, 33, device="cuda")[:, 1:]),
              lambda: mk.layer_norm_backward(x, None, st, x,
                                             workspace=torch.empty(16, device="cuda", dtype=torch.uint8))):
        with pytest.raises(mk.CoalesceError):
            c()


@pytest.mark.parametrize("types", TYPES, ids="-".join)
def test_norm_backward_of_few_rows(types):
    # one workgroup writes the sums, and one row or column more takes two launches
    dt, sdt = DT[types[0]], DT[types[1]]
    for j, (M, N) in enumerate([(8, 1023), (8, 1024), (9, 1024), (8, 1), (1, 1025), (1, 2047), (1, 2048), (1, 2049),
                                (2, 2048), (8, 301), (9, 301)]):
        progress("few rows %s %s" % (types, (M, N)))
        gen, w, _, S, _ = setup(M, N, dt, sdt, j, 3)
        dy = ref.rows(gen, M, N, dt)
        _, (mean, rstd) = mk.layer_norm_train(S, w, out_dtype=dt)
        for gd in (dt, torch.float32):
            g = mk.layer_norm_backward(S, w, (mean, rstd), dy, grad_dtype=gd)
            r = ref.norm_backward(S, w, mean, rstd, dy, None, (0.0, 0, 0), dt, sdt, gd)
            for name in ("dx", "dweight", "dbias"):
                ref.check(getattr(g, name), r[name], "%s %s" % (name, (M, N)))
