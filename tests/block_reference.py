"""64-bit references of layer norm and dropout with elementwise error bounds
(test infrastructure; numpy and plain torch, no code shared with the kernels).

Each function returns (value, bound) as ffn_reference does.  U = 2^-24 is half
a step of fp32.  A sum of N terms in fp32, in whatever order, is off by at most
(N - 1) U sum |t|; the bounds use min(N, DEPTH) additions along any path, DEPTH
= 96: per-thread runs of at most 16 values (of 8 N / 8192 + 8 <= 72 in rows
longer than 16384 up to 2^16), 6 steps within a wave, 16 waves, and the additions
of the formulas themselves.
"""
import numpy as np
import torch

from ffn_reference import U32 as U
from ffn_reference import check, f64, half_step, rounded  # noqa: F401

DEPTH = 96


def rows(gen, m, n, dtype, mean=0.0, std=1.0, pad=0, fill=float("nan")):
    """m x n normal values on the GPU in a buffer whose padding (to 16 bytes,
    and `pad` 16-byte pieces more) holds `fill`."""
    per = 16 // torch.empty((), dtype=dtype).element_size()
    ld = max(per, (n + per - 1) // per * per) + pad * per
    t = torch.full((m, ld), fill, dtype=dtype)
    t[:, :n] = (torch.randn(m, n, generator=gen) * std + mean).to(dtype)
    return t.to("cuda")[:, :n]


def space(m, n, dtype, pad=0, fill=7.0):
    """An m x n output in a buffer full of `fill`, and a check that what lies outside it still is."""
    per = 16 // torch.empty((), dtype=dtype).element_size()
    ld = max(per, (n + per - 1) // per * per) + pad * per
    t = torch.full((m, ld), fill, dtype=dtype, device="cuda")

    def untouched():
        return bool((t[:, n:] == fill).all())

    return t[:, :n], untouched


# ---------------------------------------------------------------------------
# The generator
# ---------------------------------------------------------------------------

def philox(counter, key):
    """Philox4x32-10 on arrays: counter a list of 4 and key a list of 2 uint32 arrays."""
    c = [np.asarray(x, dtype=np.uint64) for x in counter]
    k = [int(x) for x in key]
    low = np.uint64(0xFFFFFFFF)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]),
             a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return [x.astype(np.uint32) for x in c]


def kept(M, N, p, seed, offset):
    """Which elements of an M x N matrix stay, as a bool tensor on the GPU."""
    nb = (N + 3) // 4
    n, m = np.meshgrid(np.arange(nb, dtype=np.uint64), np.arange(M, dtype=np.uint64))
    o0 = np.full_like(n, offset & 0xFFFFFFFF)
    o1 = np.full_like(n, offset >> 32)
    w = np.stack(philox([n, m, o0, o1], [seed & 0xFFFFFFFF, seed >> 32]), axis=2).reshape(M, nb * 4)[:, :N]
    return torch.from_numpy(w.astype(np.int64) >= round(p * 2 ** 32)).to("cuda")


def dropped(v, e, p, seed, offset):
    """(value, bound) of a matrix known to within e after its dropout: the scale
    is rounded, and the product."""
    if round(p * 2 ** 32) == 0:
        return v, e
    k = kept(v.shape[0], v.shape[1], p, seed, offset)
    s = 1.0 / (1.0 - p) if p < 1 else 0.0
    w = torch.where(k, v * s, torch.zeros_like(v))
    # (the kept values alone: a dropped NaN is 0)
    return w, torch.where(k, e * s * (1 + 2 * U) + 2 * U * w.abs(), torch.zeros_like(w))


def dropout(x, R, p, seed, offset, dtype):
    v, e = dropped(f64(x), torch.zeros_like(f64(x)), p, seed, offset)
    if R is not None:
        v = v + f64(R)
        e = e + U * v.abs()
    return v, rounded(v, e, dtype)


# ---------------------------------------------------------------------------
# Layer norm
# ---------------------------------------------------------------------------

def norm(x, R, w, b, eps, mask, dt, sdt):
    """dict of (value, bound): y, sum, mean, rstd.  mask: (p, seed, offset)."""
    if R is None:
        s, es = f64(x), torch.zeros_like(f64(x))
    else:
        s, es = dropped(f64(x), torch.zeros_like(f64(x)), *mask)
        s = s + f64(R)
        es = es + U * s.abs()
    N = s.shape[1]
    depth = min(N, DEPTH) + 2
    mean = s.mean(1, keepdim=True)
    em = es.mean(1, keepdim=True) + depth * U * (s.abs() + es).mean(1, keepdim=True)
    d = s - mean
    ed = es + em + U * (d.abs() + es + em)
    var = d.square().mean(1, keepdim=True)
    ev = (2 * d.abs() * ed + ed * ed).mean(1, keepdim=True)
    ev = ev + depth * U * (var + ev)
    eps32 = float(np.float32(eps))
    rstd = 1 / torch.sqrt(var + eps32)
    # the root of a value known to within ev, its reciprocal and the sum with eps rounded
    hi = 1 / torch.sqrt(torch.clamp(var - ev, min=0) + eps32)
    lo = 1 / torch.sqrt(var + ev + eps32)
    er = torch.maximum(hi - rstd, rstd - lo) + 3 * U * hi
    t = d * rstd
    et = ed * rstd + d.abs() * er + ed * er + U * (t.abs() + ed * hi)
    W = f64(w)[None, :] if w is not None else torch.ones((), dtype=torch.float64, device=s.device)
    y = t * W + (f64(b)[None, :] if b is not None else 0.0)
    ey = et * W.abs() + U * (y.abs() + et * W.abs())
    return {"y": (y, rounded(y, ey, dt)), "sum": (s, rounded(s, es, sdt)), "mean": (mean[:, 0], em[:, 0]),
            "rstd": (rstd[:, 0], er[:, 0])}


def norm_backward(s, w, mean, rstd, dy, dsum, mask, dt, sdt, gdt):
    """dict of (value, bound): dx, dbranch, dweight, dbias."""
    M, N = s.shape
    depth = min(N, DEPTH) + 2
    r = f64(rstd)[:, None]
    dev = f64(s) - f64(mean)[:, None]
    xh = dev * r
    ex = 2.1 * U * xh.abs()
    dy = f64(dy)
    W = f64(w)[None, :] if w is not None else torch.ones((), dtype=torch.float64, device=dy.device)
    g = dy * W
    eg = U * g.abs()
    c1, c2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    e1 = depth * U * (g.abs() + eg).mean(1, keepdim=True) + eg.mean(1, keepdim=True)
    p = g.abs() * ex + eg * xh.abs() + eg * ex
    e2 = p.mean(1, keepdim=True) + depth * U * ((g * xh).abs() + p).mean(1, keepdim=True)
    inner = g - c1 - xh * c2
    # g - c1 and the product with xh, one rounding each (of whichever is formed first)
    ei = eg + e1 + ex * c2.abs() + e2 * xh.abs() + ex * e2 + U * (2 * g.abs() + 2 * c1.abs() + 2 * (xh * c2).abs())
    ds = r * inner
    e = r * ei + U * (ds.abs() + r * ei)
    if dsum is not None:
        ds = ds + f64(dsum)
        e = e + U * (ds.abs() + e)
    db = dropped(ds, e, *mask)
    terms = (dy * xh).abs()
    dw = (dy * xh).sum(0)
    ew = (dy.abs() * ex).sum(0) + (M + 2) * U * (terms + dy.abs() * ex).sum(0)
    dbias = dy.sum(0)
    eb = (M + 2) * U * dy.abs().sum(0)
    return {"dx": (ds, rounded(ds, e, sdt)), "dbranch": (db[0], rounded(*db, dt)),
            "dweight": (dw, rounded(dw, ew, gdt)), "dbias": (dbias, rounded(dbias, eb, gdt))}
