"""The norm's backward where every workgroup takes several rows in turn, in each of its
forms: what it keeps from row to row (the next row's loads, the two places of the
exchange, the column sums in registers and in LDS) and the ranges of rows of long rows,
against 64-bit references."""
import pytest
import torch

import block_reference as ref
import mlp_megakernel_amd as mk
from helpers import progress

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
# a wave per row, four to a workgroup, then a workgroup per row (768 of them at once; 512 of an fp32 stream with 16
# columns per thread; 256 beyond 4096 columns), each for at least two turns and a part of a third; and rows longer
# than the registers, whose columns are summed over several ranges of rows
SHAPES = [(6500, 40), (6301, 701), (1700, 1500), (1701, 2731), (1537, 4096), (801, 4100), (600, 8200), (515, 16384),
          (200, 16392), (70, 20001)]


@pytest.mark.parametrize("types", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32"), ("f32", "f32")],
                         ids="-".join)
@pytest.mark.parametrize("shape", SHAPES, ids="x".join(["%d"] * 2).__mod__)
def test_rows_in_turn(shape, types):
    M, N = shape
    dt, sdt = DT[types[0]], DT[types[1]]
    progress("rows in turn %s %s" % (shape, types))
    gen = torch.Generator().manual_seed(M + N)
    w = (1 + 0.3 * torch.randn(N, generator=gen)).to(dt).cuda()
    # rows of many means and sizes, so that none can stand for another
    S = ref.rows(gen, M, N, sdt, std=1.5)
    S += torch.linspace(-2, 2, M, device="cuda", dtype=sdt)[:, None]
    S *= (1 + 0.5 * (torch.arange(M, device="cuda") % 7)).to(sdt)[:, None]
    dy, dsum = ref.rows(gen, M, N, dt, pad=1), ref.rows(gen, M, N, sdt)
    _, stats = mk.layer_norm_train(S, w, out_dtype=dt)
    for p, ds, gd in ((0.25, dsum, torch.float32), (0.0, None, dt)):
        dx, ux = ref.space(M, N, sdt, pad=1)
        db, ub = ref.space(M, N, dt)
        g = mk.layer_norm_backward(S, w, stats, dy, ds, p, 5, 9, want_dbranch=True, grad_dtype=gd, dx=dx, dbranch=db)
        r = ref.norm_backward(S, w, *stats, dy, ds, (p, 5, 9), dt, sdt, gd)
        for name in ("dx", "dbranch", "dweight", "dbias"):
            ref.check(getattr(g, name), r[name], name)
        assert ux() and ub()
