"""64-bit references of the feed-forward operators with elementwise error
bounds (test infrastructure; plain torch, no code shared with the kernels).

Every function returns (value, bound): the operator's value in fp64 from the
inputs as they are, and how far a correct implementation may be from it, per
element.  The bounds count

* a product accumulated in fp32 in any order: (K + 2) 2^-24 sum_k |a_k b_k|
  (each of the K - 1 additions and, for MFMA's internal steps, the products
  rounded once);
* a rounding to a type of step eps: half a step relative to the value,
  eps / 2 |v|, or half the spacing of the subnormals near zero;
* the activations in fp32: see ACT_ERR.
"""
import math

import torch

U32 = 2.0 ** -24

# |act(z) as the kernels evaluate it - act(z)| <= a + r |act(z)| for an exact z.
#  * gelu: the documented absolute error of the fitted rational, 8.7e-7 (fp32
#    results and the backward) or 2.1e-5 (16-bit results), scaled by |z| above 1.
#  * silu, softplus and the sigmoid: the hardware exponential, logarithm and
#    reciprocal are good to 1 ulp (2^-23); the exponent's argument z log2(e) is
#    rounded, which moves e^-z by |z| 2^-24 relative; 8 ulp covers |z| <= 8 and
#    the sigmoid's own factor covers beyond (its error there is e^-|z| |z| 2^-24).
#    Softplus below -15 loses what 1 + t loses: half an ulp of 1.
ACT_ABS = {"none": 0.0, "relu": 0.0, "silu": 1e-7, "softplus": 2.5e-7, "gelu": 8.7e-7}
ACT_REL = {"none": 0.0, "relu": 0.0, "silu": 2.0 ** -20, "softplus": 2.0 ** -20, "gelu": 2.0 ** -21}
GELU16_ABS = 2.1e-5


def f64(t):
    return t.detach().to(torch.float64)


def half_step(v, dtype):
    """Largest error of rounding v to dtype."""
    fi = torch.finfo(dtype)
    return torch.clamp(v.abs(), min=fi.tiny) * (fi.eps / 2)


def act(z, name):
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2.0))
    if name == "softplus":
        return torch.logaddexp(z, torch.zeros_like(z))
    if name == "relu":
        return torch.clamp(z, min=0)
    return z


def act_grad(z, name):
    if name == "silu":
        s = torch.sigmoid(z)
        return s + z * s * (1 - s)
    if name == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2.0)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "softplus":
        return torch.sigmoid(z)
    if name == "relu":
        return (z > 0).to(z.dtype)
    return torch.ones_like(z)


# sup |act''| bounds how an error of z moves act(z) beyond the first order; the
# derivatives themselves are at most 1.13 (gelu) and 1.1 (silu).
SLOPE = {"none": 1.0, "relu": 1.0, "silu": 1.1, "softplus": 1.0, "gelu": 1.13}


def act_bound(z, dz, name, out16):
    """(act(z), bound) for a z known to within dz."""
    f = act(z, name)
    a = GELU16_ABS if name == "gelu" and out16 else ACT_ABS[name]
    return f, SLOPE[name] * dz + a * torch.clamp(z.abs(), min=1.0) + ACT_REL[name] * f.abs()


def preact(A, B, bias):
    A, B = f64(A), f64(B)
    K = A.shape[1]
    z, s = A @ B, A.abs() @ B.abs()
    if bias is not None:
        z, s = z + f64(bias), s + f64(bias).abs()
    return z, (K + 2) * U32 * s


def rounded(v, e, dtype):
    """Bound of a value known to within e, rounded to dtype."""
    return e + half_step(v.abs() + e, dtype)


def gated(A, Bg, Bu, bg, bu, name, out_dtype):
    (zg, eg), (zu, eu) = preact(A, Bg, bg), preact(A, Bu, bu)
    f, ef = act_bound(zg, eg, name, out_dtype != torch.float32)
    v = f * zu
    e = f.abs() * eu + zu.abs() * ef + ef * eu + U32 * v.abs()
    return v, rounded(v, e, out_dtype), (zg, rounded(zg, eg, A.dtype)), (zu, rounded(zu, eu, A.dtype))


def residual(A, B, bias, R, name, out_dtype):
    z, ez = preact(A, B, bias)
    f, ef = act_bound(z, ez, name, out_dtype != torch.float32)
    v = f + (f64(R) if R is not None else 0.0)
    e = ef + U32 * (f.abs() + v.abs())
    return v, rounded(v, e, out_dtype), (z, rounded(z, ez, A.dtype))


def _dz(dY, zg, zu, name):
    """((dz of the activated side), (dz of the other) or None), each (value, bound) before rounding."""
    dY, zg = f64(dY), f64(zg)
    g = act_grad(zg, name)
    # derivative: the sigmoid or the cdf and a few fp32 operations on values up
    # to |z| + 1 in size
    eg = 0.0 if name in ("none", "relu") else (2e-6 if name == "gelu" else 1e-6) * torch.clamp(zg.abs(), min=1.0)
    if zu is None:
        v = dY * g
        return (v, dY.abs() * eg + 2 * U32 * v.abs()), None
    zu = f64(zu)
    f, ef = act_bound(zg, torch.zeros_like(zg), name, False)
    a, b = dY * zu * g, dY * f
    return (a, (dY * zu).abs() * eg + 3 * U32 * a.abs()), (b, dY.abs() * ef + 2 * U32 * b.abs())


def backward(A, Bs, Zs, dY, name, grad_dtype):
    """dict of (value, bound): dA, dB[i], dbias[i]."""
    dt = A.dtype
    gated_ = len(Bs) == 2
    if gated_:
        dz = list(_dz(dY, Zs[0], Zs[1], name))
    elif name == "none":
        dz = [(f64(dY), torch.zeros_like(f64(dY)))]
    else:
        dz = [_dz(dY, Zs[0], None, name)[0]]
    M, N = dY.shape
    out = {"dB": [], "dbias": []}
    As = f64(A)
    dA, eA = 0.0, 0.0
    for B, (v, e) in zip(Bs, dz):
        er = rounded(v, e, dt)
        if not gated_ and name == "none" and dY.dtype == dt:
            er = e  # dZ is dY itself
        Bf = f64(B)
        dA = dA + v @ Bf.t()
        eA = eA + er @ Bf.abs().t() + (len(Bs) * N + 2) * U32 * ((v.abs() + er) @ Bf.abs().t())
        w = As.t() @ v
        ew = As.abs().t() @ er + (M + 2) * U32 * (As.abs().t() @ (v.abs() + er))
        out["dB"].append((w, rounded(w, ew, grad_dtype)))
        s = v.sum(0)
        es = e.sum(0) + (M + 2) * U32 * (v.abs() + e).sum(0)
        out["dbias"].append((s, rounded(s, es, grad_dtype)))
    out["dA"] = (dA, rounded(dA, eA, dt))
    return out


def check(got, ref, what):
    """Assert |got - value| <= bound everywhere; non-finite values only where the reference has them."""
    v, e = ref
    g = f64(got)
    assert g.shape == v.shape, "%s: shape %s, not %s" % (what, tuple(g.shape), tuple(v.shape))
    if g.numel() == 0:
        return
    bad = ~((g - v).abs() <= e)
    if bool(bad.any()):
        i = int(torch.where(bad, (g - v).abs() / e, torch.zeros_like(e)).nan_to_num(nan=float("inf")).argmax())
        raise AssertionError("%s: %d of %d values out of bounds; value %d is %r, not %r, allowed %.3g" % (
            what, int(bad.sum()), bad.numel(), i, float(g.flatten()[i]), float(v.flatten()[i]),
            float(e.flatten()[i])))
