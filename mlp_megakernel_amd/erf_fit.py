"""Derivation of the rational erf approximation used by the GELU epilogue.

GELU(z) = 0.5 z (1 + erf(z / sqrt 2)) needs erf in fp32 on every GEMM output.
The kernels evaluate

    erf(z / sqrt 2) ~= zc * P(zc^2) / Q(zc^2),  zc = clamp(z, -4 sqrt 2, 4 sqrt 2)

with P of degree 5 and Q of degree 5 (Q(0) = 1) in zc^2.  Beyond |z| = 4 sqrt 2
erf(z / sqrt 2) is +-1 to within 2^-26, so the clamp is exact in fp32.  The
coefficients below were fitted here by linearised least squares on the
relative error of erf(z/sqrt2)/z (Loeb's linearisation, P - f (Q - 1) = f),
with Lawson's iteratively reweighted scheme driving the fit toward the
minimax error; every coefficient comes out positive, so the Horner
evaluation has no cancellation.  Result: 2.5e-8 relative error in fp64 on
the fit interval; 3.3e-7 absolute on erf and 8.7e-7 on GELU (relative, floor
1) when evaluated in fp32 with FMAs and a 1-ulp reciprocal.

A second, shorter fit (P of degree 3, Q of degree 4, same method) serves
the epilogues whose output is bf16 or fp16: 5.1e-6 relative error in fp64,
2.1e-5 absolute on GELU in fp32 -- under 0.03 of an output ulp at |y| = 1
(bf16 ulp 2^-7, fp16 2^-10) -- for 13 VALU operations instead of 16.

Both have absolute errors: far left, where GELU goes to zero faster than
exp(-z^2 / 2), they leave multiples of 2^-24 |z|.  That does where the result is
what is stored; the feed-forward operators multiply it (gated product) or add to
it, so they take the normal distribution's tail with a relative error instead:

    Phi(-t) = exp(-t^2 / 2) w(t),  w(t) = erfcx(t / sqrt 2) / 2 ~= P(t) / Q(t),  0 <= t <= 13.5

(beyond, exp(-t^2 / 2) is below the smallest fp32 number).  P of degree 4, Q of
degree 5 in t, fitted the same way: 5.1e-9 relative error in fp64, all
coefficients positive.  GELU(z) = z Phi(z), Phi(z) = 1 - Phi(-z) for z > 0, is
then good to (18 + 1.25 z^2) 2^-24 relative in fp32: nine Horner steps, the two
leading coefficients, a reciprocal and an exponential of 1 ulp, three products,
and the exponent, rounded three times (z^2, the constant, their product).

    python -m mlp_megakernel_amd.erf_fit      # refits and prints the tables
"""
import numpy as np


def fit(npq: int = 6, nq: int = 5, c: float = 4.0 * np.sqrt(2.0), iters: int = 80):
    from scipy.special import erf
    z = np.cos(np.linspace(0, np.pi, 8000)) * 0.5 * c + 0.5 * c
    z = np.concatenate([z, np.linspace(0, c, 8000)])
    z = z[z > 1e-6]
    u = z * z
    f = erf(z / np.sqrt(2.0)) / z
    Q = np.ones_like(u)
    w = np.ones_like(u)
    for _ in range(iters):
        cols = [u ** i for i in range(npq)] + [-f * u ** j for j in range(1, nq + 1)]
        A = np.stack(cols, 1) / (f * Q)[:, None]
        b = f / (f * Q)
        sw = np.sqrt(w)
        sol, *_ = np.linalg.lstsq(A * sw[:, None], b * sw, rcond=None)
        p = sol[:npq]
        q = np.concatenate([[1.0], sol[npq:]])
        Qn = np.polyval(q[::-1], u)
        err = np.abs(np.polyval(p[::-1], u) / Qn - f) / f
        w = w * (err / err.max() + 1e-3)
        w /= w.mean()
        Q = Qn
    return p, q, float(err.max())


def fit_tail(npq: int = 5, nq: int = 5, c: float = 13.5, iters: int = 300):
    """(P, Q, largest relative error) of w(t) on [0, c]."""
    from scipy.special import erfcx
    t = np.concatenate([0.5 * c * (1.0 + np.cos(np.linspace(0, np.pi, 8000))), np.linspace(0, c, 8000),
                        np.linspace(0, 4, 4000)])
    f = 0.5 * erfcx(t / np.sqrt(2.0))
    Q, w, best = np.ones_like(t), np.ones_like(t), None
    for _ in range(iters):
        cols = [t ** i for i in range(npq)] + [-f * t ** j for j in range(1, nq + 1)]
        A = np.stack(cols, 1) / (f * Q)[:, None]
        scale = np.abs(A).max(0)
        sw = np.sqrt(w)
        sol = np.linalg.lstsq(A / scale * sw[:, None], sw / Q, rcond=None)[0] / scale
        p, q = sol[:npq], np.concatenate([[1.0], sol[npq:]])
        Q = np.polyval(q[::-1], t)
        err = np.abs(np.polyval(p[::-1], t) / Q - f) / f
        if best is None or err.max() < best[2]:
            best = p, q, float(err.max())
        w = w * (err / err.max() + 1e-3)
        w /= w.mean()
    return best


if __name__ == "__main__":
    for npq, nq, what in ((6, 5, "fp32 outputs"), (4, 4, "16-bit outputs")):
        p, q, e = fit(npq, nq)
        print("%s: max relative error (fp64): %.3e" % (what, e))
        print("P:", ", ".join("%.9ef" % v for v in p))
        print("Q:", ", ".join("%.9ef" % v for v in q))
    p, q, e = fit_tail()
    print("tail: max relative error (fp64): %.3e" % e)
    print("P:", ", ".join("%.9ef" % v for v in p))
    print("Q:", ", ".join("%.9ef" % v for v in q))
