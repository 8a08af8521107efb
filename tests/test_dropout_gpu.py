"""Dropout on the GPU against the generator's definition (block_reference.py) and
its 64-bit values: every type, odd extents, in place, seeds in device memory."""
import pytest
import torch

import block_reference as ref
import mlp_megakernel_amd as mk
from helpers import progress

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32"), ("f32", "f32")]
SHAPES = [(1, 1), (3, 3), (257, 4), (2, 9), (40, 63), (33, 512), (5, 2047), (3, 2049), (7, 4100), (1001, 2731)]


@pytest.mark.parametrize("types", TYPES, ids="-".join)
@pytest.mark.parametrize("p", [0.0, 1e-4, 0.1, 0.5, 0.999, 1.0])
def test_dropout(types, p):
    dt, odt = DT[types[0]], DT[types[1]]
    for j, (M, N) in enumerate(SHAPES):
        progress("dropout %s %s %s" % (types, p, (M, N)))
        gen = torch.Generator().manual_seed(31 * M + N)
        seed, offset = (0xFEDCBA9876543210 + j) & 0xFFFFFFFFFFFFFFFF, (j << 40) + 3
        x, R = ref.rows(gen, M, N, dt, pad=j % 2), ref.rows(gen, M, N, odt, pad=1)
        out, untouched = ref.space(M, N, odt, pad=j % 3)
        ref.check(mk.dropout(x, p, seed, offset, residual=R, out=out), ref.dropout(x, R, p, seed, offset, odt),
                  "sum %s" % ((M, N),))
        assert untouched()
        y = mk.dropout(x, p, seed, offset, out=mk.aligned_empty(M, N, odt))
        ref.check(y, ref.dropout(x, None, p, seed, offset, odt), "alone %s" % ((M, N),))
        if p >= 0.1:
            assert bool((y[~ref.kept(M, N, p, seed, offset)] == 0).all())
        # in place of the residual, and of x; the gradient is the same operation
        R2, untouched = ref.space(M, N, odt)
        R2.copy_(R)
        assert torch.equal(mk.dropout(x, p, seed, offset, residual=R2, out=R2), out) and untouched()
        if dt == odt:
            x2, untouched = ref.space(M, N, dt)
            x2.copy_(x)
            assert torch.equal(mk.dropout_backward(x2, p, seed, offset, out=x2), y) and untouched()


def test_share_that_stays():
    # 2^22 draws: the share kept is within 5 deviations of 1 - p
    x = torch.ones(2048, 2048, device="cuda")
    for p in (0.01, 0.1, 0.5, 0.9):
        n = float((mk.dropout(x, p, 17) != 0).sum())
        assert abs(n / 2 ** 22 - (1 - p)) <= 5 * (p * (1 - p) / 2 ** 22) ** 0.5


def test_mask_goes_by_the_place_alone():
    gen = torch.Generator().manual_seed(2)
    x = ref.rows(gen, 70, 300, torch.float32)
    a = mk.dropout(x, 0.3, 5) != 0
    assert torch.equal(mk.dropout(x[:40, :123], 0.3, 5) != 0, a[:40, :123])
    assert torch.equal(mk.dropout(mk.aligned_copy(x.bfloat16()), 0.3, 5) != 0, a)
    for other in (mk.dropout(x, 0.3, 6), mk.dropout(x, 0.3, 5, 1), mk.dropout(x, 0.3, 5 + 2 ** 32),
                  mk.dropout(x, 0.3, 5, 2 ** 32)):
        assert not torch.equal(other != 0, a)
    assert torch.equal(mk.dropout(x, 0.3, 5 - 2 ** 64) != 0, a)  # (as the 64 bits that it is)
    # the fused sum takes the same mask
    _, s = mk.add_layer_norm(x, torch.zeros_like(x), p=0.3, seed=5)
    assert torch.equal(s, mk.dropout(x, 0.3, 5))


def test_dropped_values_are_zero_whatever_they_were():
    x = torch.full((64, 64), float("nan"), device="cuda", dtype=torch.float16)
    x[::2] = float("inf")
    y = mk.dropout(x, 0.5, 1)
    k = ref.kept(64, 64, 0.5, 1, 0)
    assert bool((y[~k] == 0).all()) and not bool(y[k].isfinite().any())
    assert bool((mk.dropout(x, 1.0, 1) == 0).all())


def test_seed_in_device_memory_is_read_by_the_kernel():
    gen = torch.Generator().manual_seed(3)
    x = ref.rows(gen, 50, 100, torch.bfloat16)
    both = torch.tensor([1, 0], device="cuda")
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mk.dropout(x, 0.4, both)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        y = mk.dropout(x, 0.4, both)
    for seed, offset in ((1, 0), (2, 0), (2, 5), (-3, 2 ** 40)):
        both.copy_(torch.tensor([seed, offset]))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, mk.dropout(x, 0.4, seed, offset))
    s2 = torch.cuda.Stream()
    s2.wait_stream(torch.cuda.current_stream())
    z = mk.dropout(x, 0.4, both, stream=s2)
    s2.synchronize()
    assert torch.equal(z, y)


def test_far_rows():
    M, N = (1 << 21) + 3, 1030
    x = torch.ones(M, 1032, device="cuda", dtype=torch.bfloat16)[:, :N]
    y = mk.dropout(x, 0.5, 9)
    # rows at the end and in the middle against the generator
    for m0 in (M - 3, 1 << 20):
        n, m = torch.meshgrid(torch.arange(N), torch.arange(m0, m0 + 3), indexing="xy")
        w = ref.philox([(n // 4).numpy(), m.numpy(), 0 * m.numpy(), 0 * m.numpy()], [9, 0])
        word = torch.stack([torch.from_numpy(v.astype("int64")) for v in w], 2).gather(2, (n % 4)[:, :, None])[:, :, 0]
        assert torch.equal((y[m0:m0 + 3] != 0).cpu(), word >= 2 ** 31)


def test_refusals():
    x = torch.zeros(4, 32, device="cuda", dtype=torch.bfloat16)
    for c in (lambda: mk.dropout(x, 0.1, 1, residual=x.half()), lambda: mk.dropout(x.float(), 0.1, 1, residual=x),
              lambda: mk.dropout(x, 0.1, 1, out=x[:3]), lambda: mk.dropout(x.int(), 0.1, 1),
              lambda: mk.dropout(x, 0.1, torch.zeros(2, device="cuda")), lambda: mk.dropout(x.cpu(), 0.1, 1)):
        with pytest.raises(ValueError):
            c()
    for c in (lambda: mk.dropout(x, -0.1, 1), lambda: mk.dropout(x, 1.1, 1), lambda: mk.dropout(x, float("nan"), 1),
              lambda: mk.dropout(x[:2], 0.1, 1, out=x[1:3])):
        with pytest.raises(mk.CoalesceError):
            c()
    assert mk.dropout(x[:0], 0.1, 1).shape == (0, 32)
