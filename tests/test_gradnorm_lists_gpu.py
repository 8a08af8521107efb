"""Lists of gradients as callers have them: generators whose tensors nobody else
holds, on the current stream and on another."""
import math

import pytest
import torch

import mlp_megakernel_amd as mk

pytestmark = pytest.mark.gpu


def _values(n=12):
    gen = torch.Generator(device="cuda").manual_seed(1)
    # sizes from that of the norm itself up, so that freed blocks fit what a call makes
    return [torch.randn(1 << (i + 2), generator=gen, device="cuda") for i in range(n)]


@pytest.mark.parametrize("norm_type", [2, math.inf])
def test_temporaries_of_a_generator(norm_type):
    xs = _values()
    want = torch.stack([(2.0 * x.double()).norm(norm_type) for x in xs]).norm(norm_type)
    torch.cuda.synchronize()
    for _ in range(3):
        n = mk.grad_norm((2.0 * x for x in xs), norm_type=norm_type)
        assert abs(float(n) - float(want)) <= 2.0 ** -23 * float(want)
        outs = [torch.empty_like(x) for x in xs]
        n2 = mk.clip_grad_norm((2.0 * x for x in xs), 1.0, norm_type=norm_type, out=(o for o in outs))
        assert torch.equal(n, n2)
        c = 1.0 / (want + 1e-6)
        for x, o in zip(xs, outs):
            # c and the product, each rounded to fp32
            v = 2.0 * x.double() * c
            assert bool(((o.double() - v).abs() <= 2.0 ** -23 * v.abs()).all())


def test_temporaries_of_a_generator_on_another_stream():
    # made late on the current stream, read on the other, their blocks taken again at once
    xs = _values()
    want = torch.stack([(2.0 * x.double()).norm() for x in xs]).norm()
    side = torch.cuda.Stream()
    for handle in (side, side.cuda_stream):
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)
        n = mk.grad_norm((2.0 * x for x in xs), stream=handle)
        again = [torch.full_like(x, 1e30) for x in xs]
        torch.cuda.synchronize()
        assert abs(float(n) - float(want)) <= 2.0 ** -23 * float(want)
        del again


def test_generator_of_parameters_gradients():
    m = mk.GatedFFN(64, 128)
    x = torch.randn(10, 64, device="cuda", dtype=torch.bfloat16)
    m(x).float().sum().backward()
    want = torch.cat([p.grad.double().flatten() for p in m.parameters()]).norm()
    n = mk.clip_grad_norm((p.grad for p in m.parameters()), 0.25)
    assert abs(float(n) - float(want)) <= 2.0 ** -23 * float(want)
    assert float(mk.grad_norm(p.grad for p in m.parameters())) <= 0.26
