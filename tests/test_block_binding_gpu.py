"""The two ways into layer norm, dropout, quantisation and the 8-bit products, through
compiled code and through the checks in Python: the same results, and the same refusals."""
import importlib

import pytest
import torch

import block_reference as ref
import mlp_megakernel_amd as mk

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
norm_py = importlib.import_module("mlp_megakernel_amd.norm")
int8_py = importlib.import_module("mlp_megakernel_amd.int8")


def flat(r):
    if r is None or isinstance(r, torch.Tensor):
        return [r]
    return [t for v in r for t in flat(v)]


class Ways:
    """Runs a call both ways; counts how often compiled code answered."""

    def __init__(self, monkeypatch):
        self.short, self.answers, self.on = norm_py._short, 0, True
        for m in (norm_py, int8_py):
            monkeypatch.setattr(m, "_short", self.call)

    def call(self, *a):
        got = self.short(*a) if self.on else None
        self.answers += got is not None
        return got

    def both(self, call):
        self.on, before = True, self.answers
        quick = flat(call())
        assert self.answers > before, "compiled code did not take the call"
        self.on = False
        slow = flat(call())
        assert len(quick) == len(slow)
        for a, b in zip(quick, slow):
            assert (a is None) == (b is None)
            if a is not None:
                assert a.dtype is b.dtype and a.shape == b.shape and a.stride() == b.stride() and torch.equal(a, b)


@pytest.fixture
def ways(monkeypatch):
    return Ways(monkeypatch)


@pytest.mark.parametrize("M,N", [(1, 5), (7, 64), (33, 301), (300, 1001), (0, 40)])
@pytest.mark.parametrize("types", [(BF, BF, BF, F32), (BF, F32, F32, BF), (torch.float16, F32, torch.float16, F32)])
def test_norm_and_dropout(ways, M, N, types):
    dt, st, wt, gt = types
    gen = torch.Generator().manual_seed(M + N)
    r = lambda t, pad=0: ref.rows(gen, M, N, t, pad=pad)  # noqa: E731
    x, s, res, dy, ds = r(dt), r(st, 1), r(st), r(dt, 1), r(st)
    w, b = (torch.randn(N, generator=gen).to(wt).cuda() for _ in range(2))
    stats = mk.layer_norm_train(s, w, b, out_dtype=dt)[1]
    seed = torch.tensor([5, 9], device="cuda")
    ways.both(lambda: mk.layer_norm_train(s, w, b, out_dtype=dt))
    ways.both(lambda: mk.add_layer_norm_train(x, res, w, b, p=0.3, seed=seed))
    ways.both(lambda: mk.add_layer_norm(x, res, w, None, p=0.3, seed=5, offset=9))
    ways.both(lambda: mk.layer_norm_backward(s, w, stats, dy, ds, 0.3, seed, want_dbranch=True, grad_dtype=gt))
    ways.both(lambda: mk.layer_norm_backward(s, w, stats, dy, None, 0.3, 5, 9, want_dx=0, want_dbranch=1,
                                             dx=torch.full_like(s, 3)))
    ways.both(lambda: mk.layer_norm_backward(s, None, stats, dy, want_dx=False, want_dweight=False))
    ways.both(lambda: mk.layer_norm_backward(s, w, stats, dy, want_dweight=False, want_dbias=False,
                                             dx=ref.space(M, N, st)[0]))
    ways.both(lambda: mk.layer_norm_backward(s, w, stats, dy, ds, workspace=torch.empty(1 << 24, dtype=torch.uint8,
                                                                                         device="cuda")))
    ways.both(lambda: mk.dropout(x, 0.3, seed, residual=res))
    ways.both(lambda: mk.dropout(x, 0.3, 5, 9))


def test_the_masks_seed_is_read_alike(ways):
    # 64 bits, modulo 2^64; both in device memory or both not
    x = torch.ones(40, 64, device="cuda")
    for seed, offset in ((-1, 3), (2 ** 64 - 1, 3), (2 ** 64 + 5, -2), (True, 0)):
        ways.both(lambda: mk.dropout(x, 0.5, seed, offset))
    wrap = lambda v: v - 2 ** 64 if v >= 2 ** 63 else v  # noqa: E731
    ways.on = True
    for seed, offset in ((2 ** 64 - 1, 3), (5, 2 ** 63 + 1)):
        there = torch.tensor([wrap(seed), wrap(offset)], device="cuda")
        assert torch.equal(mk.dropout(x, 0.5, there), mk.dropout(x, 0.5, seed, offset))


@pytest.mark.parametrize("M,N,K", [(1, 24, 16), (40, 301, 203), (100, 64, 5000)])
def test_8_bits(ways, M, N, K):
    gen = torch.Generator().manual_seed(N)
    x, W = ref.rows(gen, M, K, BF), ref.rows(gen, K, N, BF)
    q, s = mk.quantize_rows(x)
    B, sb = mk.quantize_columns(W)
    res, bias = ref.rows(gen, M, N, F32), torch.randn(N, generator=gen).cuda()
    ways.both(lambda: mk.quantize_rows(x))
    ways.both(lambda: mk.quantize_columns(W))
    ways.both(lambda: mk.gemm_int8(q, B, s, sb, bias, res, "gelu"))
    ways.both(lambda: mk.gemm_int8(q, B, s, sb))
    ways.both(lambda: mk.gated_gemm_int8(q, B, B, s, sb, sb, bias, None, out_dtype=torch.float16))


@pytest.mark.parametrize("quick", [True, False])
def test_refusals(ways, quick):
    ways.on = quick
    x = torch.randn(8, 64, device="cuda", dtype=BF)
    w = torch.ones(64, device="cuda", dtype=BF)
    y, stats = mk.layer_norm_train(x, w, w)
    back = lambda **kw: mk.layer_norm_backward(**{**dict(x=x, weight=w, stats=stats, dout=y), **kw})  # noqa: E731
    seed = torch.tensor([1, 2], device="cuda")
    for kw in (dict(stats=stats[:1]), dict(stats=(stats[0][:7], stats[1])), dict(dout=y[:7]), dict(dout=y.float()),
               dict(grad_dtype=torch.float16), dict(grad_dtype=torch.float64), dict(dx=x.float()), dict(dx=x[:, ::2]),
               dict(weight=w[:63]), dict(weight=w.half()), dict(dsum=x.float()), dict(x=x[0]), dict(x=x.cpu()),
               dict(seed=seed, offset=1, p=0.5), dict(seed=seed.int(), p=0.5),
               dict(workspace=torch.empty(64, 64, device="cuda").t()[:32])):
        with pytest.raises(ValueError):
            back(**kw)
    for kw in (dict(p=1.5), dict(dx=y), dict(dx=x), dict(workspace=torch.empty(16, device="cuda", dtype=torch.uint8))):
        with pytest.raises(mk.CoalesceError):
            back(**kw)
    with pytest.raises(ValueError):
        mk.dropout(x, 0.5, seed, offset=1)
    with pytest.raises(ValueError):
        mk.layer_norm(x, w, w, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        mk.layer_norm(x, w, w, out_dtype=BF, out=torch.empty(8, 64, device="cuda"))
    q, s = mk.quantize_rows(x)
    with pytest.raises(ValueError):
        mk.gemm_int8(q, q, s, s, out_dtype=BF, out=torch.empty(8, 8, device="cuda"))
    with pytest.raises(ValueError):
        mk.gemm_int8(q, q, s, s, residual=torch.empty(8, 8, device="cuda"), out_dtype=BF)
