"""Norm and clipping of matrices whose rows lie apart: the framework's own
gradients at widths that are no multiple of 16 bytes, halves of wider matrices,
narrow and very wide rows, many of them, among dense tensors.  Between the rows
stands NaN, which must neither be read into the norm nor written."""
import math

import pytest
import torch

import mlp_megakernel_amd as mk
from helpers import progress
from test_ffn_gpu import problem, rows
from test_gradnorm_gpu import check

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def apart(gen, m, n, dtype, gap, shift=0):
    """(buffer, m x n view of it): rows n + gap elements apart, `shift` elements into the buffer, NaN elsewhere."""
    buf = torch.full((m * (n + gap) + shift,), float("nan"), dtype=dtype, device="cuda")
    v = buf[shift:shift + m * (n + gap)].view(m, n + gap)[:, :n]
    v.copy_(torch.randn(m, n, generator=gen, device="cuda") * 0.3)
    return buf, v


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("norm_type", [2, math.inf])
@pytest.mark.parametrize("shapes", [[(2, 1)], [(3, 5), (100, 7)], [(1, 9), (64, 64), (33, 1000)], [(5, 40000), (2, 3)],
                                    [(3000, 13)], [(17 + i, 30 + 3 * i) for i in range(150)], [(1000, 2731), (2731, 1001)]])
def test_clip(dt, norm_type, shapes):
    d = DT[dt]
    gen = torch.Generator(device="cuda").manual_seed(len(shapes))
    for max_norm in (0.05, 1e9, 0.0):
        src = [apart(gen, m, n, d, gap=1 + i % 9, shift=i % 4) for i, (m, n) in enumerate(shapes)]
        dst = [apart(gen, m, n, d, gap=8 - i % 5, shift=i % 3) for i, (m, n) in enumerate(shapes)]
        keep = [b.clone() for b, _ in src]
        norm = mk.clip_grad_norm([v for _, v in src], max_norm, norm_type=norm_type, out=[v for _, v in dst])
        for (b, _), k in zip(src, keep):
            assert torch.equal(b.nan_to_num(nan=9.0), k.nan_to_num(nan=9.0))
        check([v for _, v in src], [v for _, v in dst], norm, max_norm, norm_type)
        for b, v in dst:
            assert int(torch.isnan(b).sum()) == b.numel() - v.numel()
        # in place, and of dense copies: the same values
        dense = [v.clone(memory_format=torch.contiguous_format) for _, v in src]
        norm2 = mk.clip_grad_norm(dense, max_norm, norm_type=norm_type)
        assert abs(float(norm) - float(norm2)) <= 2.0 ** -23 * float(norm)
        norm3 = mk.clip_grad_norm([v for _, v in src], max_norm, norm_type=norm_type)
        assert torch.equal(norm, norm3)
        for (b, v), (_, o) in zip(src, dst):
            assert torch.equal(v, o) and int(torch.isnan(b).sum()) == b.numel() - v.numel()
        assert float(mk.grad_norm([v for _, v in dst], norm_type=norm_type)) <= max(float(norm), max_norm) * 1.01
    progress("%s %s %d" % (dt, norm_type, len(shapes)))


def test_mixed_with_dense_tensors():
    gen = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s, dt=torch.float32: torch.randn(*s, generator=gen, device="cuda").to(dt)  # noqa: E731
    ts = [apart(gen, 40, 33, torch.bfloat16, 7)[1], r(1000, dt=torch.bfloat16), apart(gen, 9, 130, torch.float32, 2)[1],
          r(33, 65), r(64, 40).t(), apart(gen, 70, 3, torch.float16, 5)[1], torch.empty(0, 5, device="cuda"),
          torch.full((1, 70), float("nan"), device="cuda")[:, :0]]
    # outputs: dense for padded, padded for dense, and the same
    outs = [torch.empty(40, 33, device="cuda", dtype=torch.bfloat16), torch.empty_like(ts[1]), torch.empty_like(ts[2]),
            apart(gen, 33, 65, torch.float32, 4)[1], torch.empty_like(ts[4]), apart(gen, 70, 3, torch.float16, 1)[1],
            torch.empty_like(ts[6]), torch.empty_like(ts[7])]
    norm = mk.clip_grad_norm(ts, 1.0, out=outs)
    check(ts, outs, norm, 1.0)
    assert abs(float(mk.grad_norm(outs)) - 1.0) < 1e-2


@pytest.mark.parametrize("grad", [torch.bfloat16, torch.float32])
def test_gradients_of_the_backward_at_odd_widths(grad):
    _, A, Bs, bs = problem(70, 131, 75, torch.bfloat16, nb=2)
    gen = torch.Generator().manual_seed(1)
    _, Z = mk.gated_gemm_train(A, *Bs, *bs)
    dY = rows(gen, 70, 131, 1.0, torch.bfloat16)
    g = mk.gated_gemm_backward(A, *Bs, Z, dY, want_dbias=True, grad_dtype=grad)
    r = mk.gemm_residual_backward(A, Bs[0], dY, want_dbias=True, grad_dtype=grad)
    grads = [t for t in (*g, *r)]
    assert not g.dBg.is_contiguous()
    outs = [torch.empty_like(t) for t in grads]
    norm = mk.clip_grad_norm(grads, 0.5, out=outs)
    check(grads, outs, norm, 0.5)
    assert torch.equal(norm, mk.clip_grad_norm(grads, 0.5)) and all(torch.equal(a, b) for a, b in zip(grads, outs))


def test_halves_of_one_matrix():
    gen = torch.Generator(device="cuda").manual_seed(4)
    W = torch.randn(50, 144, generator=gen, device="cuda")
    keep = W.clone()
    norm = mk.clip_grad_norm([W[:, :72], W[:, 72:]], 1.0)
    check([keep], [W], norm, 1.0)
    for a, b in ((W[:, :73], W[:, 72:]), (W[:, 10:20], W[:, 15:16]), (W[:, :72], W[3])):
        with pytest.raises((ValueError, RuntimeError)):
            mk.clip_grad_norm([a, b], 1.0)
    with pytest.raises((ValueError, RuntimeError)):
        mk.clip_grad_norm([W[:, :72]], 1.0, out=[W[:, 60:132]])
    with pytest.raises((ValueError, RuntimeError)):   # in place with another pitch
        mk.clip_grad_norm([W.view(-1)[:50 * 72].view(50, 72)], 1.0, out=[W[:, :72]])
    for t in (W[::2, ::2], W[:, None, :].expand(50, 3, 144), W[0].expand(4, 144), torch.empty(3, 4, 8, device="cuda")[:, :, :5]):
        with pytest.raises((ValueError, RuntimeError)):
            mk.grad_norm([t])
    assert not bool(torch.isnan(W).any())


def test_captured_and_replayed():
    gen = torch.Generator(device="cuda").manual_seed(5)
    buf, v = apart(gen, 300, 77, torch.bfloat16, 3)
    dense = torch.randn(5000, generator=gen, device="cuda")
    out = [torch.empty_like(v), torch.empty_like(dense)]
    norm = torch.empty((), device="cuda")
    mk.clip_grad_norm([v, dense], 1.0, out=out, norm=norm)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mk.clip_grad_norm([v, dense], 1.0, out=out, norm=norm)
    for i in range(4):
        v.normal_(generator=gen)
        want_out = [torch.empty_like(o) for o in out]
        want = mk.clip_grad_norm([v, dense], 1.0, out=want_out)
        torch.cuda.synchronize()
        for o in out:
            o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(norm, want) and all(torch.equal(a, b) for a, b in zip(out, want_out)), i
