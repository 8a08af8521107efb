"""Layer norm and its gradients at the edges of their range: rows whose values, mean or
deviations are far from 1, against 64-bit references."""
import pytest
import torch

import block_reference as ref
import mlp_megakernel_amd as mk
from helpers import progress

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f32"), ("f32", "f32")]
# each form of the kernels, with columns of the last thread outside the row, and one that its row fills
WIDTHS = [100, 701, 1500, 2048, 3001, 5000, 9003, 16400]


def check_backward(S, w, stats, dy, dsum, mask, dt, what):
    g = mk.layer_norm_backward(S, w, stats, dy, dsum, *mask, want_dbranch=True)
    r = ref.norm_backward(S, w, *stats, dy, dsum, mask, dt, S.dtype, torch.float32)
    for name in ("dx", "dbranch", "dweight", "dbias"):
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
