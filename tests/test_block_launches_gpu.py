"""Layer norm, quantisation and dropout over more rows or elements than one
dimension of a launch holds (it counts its threads in 32 bits)."""
import pytest
import torch

import mlp_megakernel_amd as mk
from helpers import progress

pytestmark = pytest.mark.gpu

ROWS = (1 << 26) + 3  # a wave of 64 for each: 192 threads past 2^32


def values():
    x = torch.randn(4096, 8, device="cuda", dtype=torch.bfloat16).repeat(ROWS // 4096 + 1, 1)[:ROWS]
    x[-3:] = torch.arange(24, device="cuda").view(3, 8)
    return x


def test_norm_of_many_rows():
    x = values()
    g, b = (torch.randn(8, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    progress("norm of %d rows" % ROWS)
    y, stats = mk.layer_norm_train(x, g, b)
    want, want_stats = mk.layer_norm_train(x[:4096], g, b)
    tail, tail_stats = mk.layer_norm_train(x[-3:], g, b)
    for got, w, t in zip((y, *stats), (want, *want_stats), (tail, *tail_stats)):
        whole = (ROWS - 3) // 4096 * 4096
        assert bool((got[:whole].view(-1, *w.shape) == w).all())
        assert torch.equal(got[-3:], t)


def test_quantisation_of_many_rows():
    x = values()
    progress("quantisation of %d rows" % ROWS)
    q, s = mk.quantize_rows(x)
    qw, sw = mk.quantize_rows(x[:4096])
    qt, st = mk.quantize_rows(x[-3:])
    whole = (ROWS - 3) // 4096 * 4096
    assert bool((s[:whole].view(-1, 4096) == sw).all()) and torch.equal(s[-3:], st)
    assert bool((q[:whole].view(-1, 4096, 8) == qw).all()) and torch.equal(q[-3:], qt)


def test_dropout_of_many_elements():
    # 8 elements a thread: 2^32 threads of them and one row more, in place; with p = 1 every one is written
    x = torch.ones((1 << 21) + 1, 1 << 14, device="cuda", dtype=torch.float16)
    progress("dropout of %d elements" % x.numel())
    mk.dropout(x, 1.0, seed=1, offset=2, out=x)
    for part in x.split(1 << 17):
        assert not bool(part.any())
