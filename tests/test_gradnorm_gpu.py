"""GPU parity of the gradient norm and of clipping: mixed types, odd sizes and
alignments, empty tensors, many tensors, infinities and NaN, out of place and
in place, against fp64."""
import math

import pytest
import torch

import mlp_megakernel_amd as mk
from ffn_reference import half_step

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def exact(tensors, max_norm, norm_type):
    flat = [t.detach().to(torch.float64).flatten() for t in tensors]
    flat = torch.cat(flat) if flat else torch.zeros(0, dtype=torch.float64)
    n = float(flat.abs().max()) if norm_type == math.inf and flat.numel() else float(flat.norm()) if norm_type == 2 else 0.0
    c = min(1.0, max_norm / (n + 1e-6))
    return n, c


def check(tensors, outs, norm, max_norm, norm_type=2):
    n, c = exact(tensors, max_norm, norm_type)
    # the norm: fp64 sums (2^-53 a step, negligible), one rounding to fp32
    assert abs(float(norm) - n) <= 2.0 ** -24 * n + 1e-30 + 1e-12 * n, (float(norm), n)
    for i, (t, o) in enumerate(zip(tensors, outs)):
        v = t.to(torch.float64) * c
        # c rounded to fp32, one product in fp32, one rounding to the type
        e = 2 * 2.0 ** -24 * v.abs() + half_step(v, t.dtype) if c < 1.0 else torch.zeros_like(v)
        bad = ~((o.to(torch.float64) - v).abs() <= e)
        assert not bool(bad.any()), "tensor %d: %d values off" % (i, int(bad.sum()))


def packed(sizes, dtype, seed, gap=0):
    """Views into one buffer, one behind the other: only element alignment."""
    gen = torch.Generator().manual_seed(seed)
    flat = (torch.randn(sum(sizes) + gap * len(sizes) + 1, generator=gen) * 0.3).to(dtype).to("cuda")
    views, at = [], 1
    for n in sizes:
        views.append(flat[at:at + n])
        at += n + gap
    return flat, views


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("norm_type", [2, math.inf])
@pytest.mark.parametrize("sizes", [[1], [7], [0, 5, 0], [1023, 1, 64, 4097, 3, 0, 130], [300000], [128] * 250 + [70001]])
def test_clip(dt, norm_type, sizes):
    d = DT[dt]
    for max_norm in (0.05, 1e9, 0.0):
        src_flat, src = packed(sizes, d, 1 + len(sizes))
        keep = src_flat.clone()
        flat, outs = packed(sizes, d, 2, gap=3)
        flat.fill_(9.0)
        norm = mk.clip_grad_norm(src, max_norm, norm_type=norm_type, out=outs)
        assert torch.equal(src_flat, keep)
        check(src, outs, norm, max_norm, norm_type)
        assert int((flat == 9.0).sum()) >= 3 * len(sizes) + 1  # the gaps
        # the same list in place, and a second call on other buffers: the same bits
        norm2 = mk.clip_grad_norm(src, max_norm, norm_type=norm_type)
        assert torch.equal(norm, norm2)
        for a, b in zip(src, outs):
            assert torch.equal(a, b)
        assert float(mk.grad_norm(outs, norm_type=norm_type)) <= max(float(norm), max_norm) * 1.01


def test_mixed_types_and_shapes():
    gen = torch.Generator().manual_seed(5)
    ts = [torch.randn(33, 65, generator=gen).to("cuda"), torch.randn(1000, generator=gen).to(torch.bfloat16).to("cuda"),
          torch.randn(3, 5, 7, generator=gen).to(torch.float16).to("cuda"),
          torch.randn(64, 40, generator=gen).to(torch.bfloat16).to("cuda").t(), torch.tensor(2.0, device="cuda")]
    outs = [torch.empty_like(t) for t in ts]
    norm = mk.clip_grad_norm(ts, 1.0, out=outs)
    check(ts, outs, norm, 1.0)


def test_large_values_do_not_overflow():
    ts = [torch.full((1000,), 1e25, device="cuda"), torch.full((5,), 1e-30, device="cuda")]
    norm = mk.clip_grad_norm(ts, 1.0)
    assert abs(float(norm) / (1e25 * math.sqrt(1000)) - 1) < 1e-6
    assert torch.allclose(ts[0], torch.full((1000,), 1 / math.sqrt(1000), device="cuda"), rtol=1e-6)


@pytest.mark.parametrize("norm_type", [2, math.inf])
def test_nonfinite(norm_type):
    ts = [torch.ones(300, device="cuda"), torch.ones(700, device="cuda", dtype=torch.bfloat16)]
    ts[1][3] = float("nan")
    outs = [torch.empty_like(t) for t in ts]
    assert math.isnan(float(mk.clip_grad_norm(ts, 1.0, norm_type=norm_type, out=outs)))
    assert bool(torch.isnan(outs[0]).all()) and bool(torch.isnan(outs[1]).all())
    ts[1][3] = float("-inf")
    assert float(mk.clip_grad_norm(ts, 1.0, norm_type=norm_type, out=outs)) == math.inf
    assert float(outs[0].abs().sum()) == 0.0 and bool(torch.isnan(outs[1][3]))


def test_empty_list():
    assert float(mk.grad_norm([])) == 0.0 and float(mk.clip_grad_norm([], 1.0)) == 0.0
