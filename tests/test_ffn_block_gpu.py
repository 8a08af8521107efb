"""The feed-forward operators used together: the GatedFFN module against the
block written out in fp64 (values and every gradient), against differences,
a training step whose gradients are clipped, the same calls captured in a
graph and replayed, and on another stream than the current one."""
import pytest
import torch

import ffn_reference as ref
import mlp_megakernel_amd as mk

pytestmark = pytest.mark.gpu


def block64(p, x, act, residual):
    zg, zu = x @ p["Wg"], x @ p["Wu"]
    if "bg" in p:
        zg, zu = zg + p["bg"], zu + p["bu"]
    y = (ref.act(zg, act) * zu) @ p["Wd"]
    if "bd" in p:
        y = y + p["bd"]
    return x + y if residual else y


def rel(a, b):
    return float((a.to(torch.float64) - b).norm() / b.norm())


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("act,bias,residual,shape", [("silu", False, True, (3, 17, 64)), ("gelu", True, False, (130, 72)),
                                                     ("relu", True, True, (1, 100)), ("silu", True, True, (2, 33, 71))])
def test_block_matches_fp64(dt, act, bias, residual, shape):
    torch.manual_seed(0)
    D, H = shape[-1], 2 * shape[-1] + 37
    m = mk.GatedFFN(D, H, act=act, bias=bias, residual=residual, dtype=dt)
    if bias:
        for b in (m.bg, m.bu, m.bd):
            torch.nn.init.normal_(b, std=0.3)
    x = torch.randn(shape, device="cuda").to(dt).requires_grad_()
    dy = torch.randn(shape, device="cuda").to(dt)
    y = m(x)
    y.backward(dy)
    with torch.no_grad():
        assert torch.equal(m(x), y), "inference and training forward differ"
    p = {k: v.detach().to(torch.float64).requires_grad_() for k, v in m.named_parameters()}
    x64 = x.detach().to(torch.float64).requires_grad_()
    y64 = block64(p, x64, act, residual)
    y64.backward(dy.to(torch.float64))
    # Five roundings to the type lie between the inputs and any gradient (Z, H
    # or dH, dZ, the output); each moves it by at most half a step relative to
    # its operands, which stay within a factor 4 of the result in norm here
    # (relu'(z), act(z) <= |z|, unit-variance sums).
    tol = 5 * 4 * torch.finfo(dt).eps / 2
    assert rel(y, y64) <= tol
    assert rel(x.grad, x64.grad) <= tol
    for k, v in m.named_parameters():
        assert v.grad is not None and v.grad.dtype == dt and rel(v.grad, p[k].grad) <= tol, k


def test_gradient_against_differences():
    # <dY, f(W + h V) - f(W - h V)> / 2h against <dW, V>, from fp32 outputs of
    # fp16 operands: f is smooth (silu), so the difference quotient's own error
    # is O(h^2); the quotient and the gradient agree to their roundings
    torch.manual_seed(1)
    M, N, K = 40, 48, 56
    A, Bg, Bu = (torch.randn(s, device="cuda").half() * f for s, f in (((M, K), 1.0), ((K, N), 0.15), ((K, N), 0.15)))
    dY = torch.randn(M, N, device="cuda")
    _, Z = mk.gated_gemm_train(A, Bg, Bu)
    g = mk.gated_gemm_backward(A, Bg, Bu, Z, dY)
    h = 2.0 ** -6
    f = lambda g_, u_: float((mk.gated_gemm(A, g_, u_, out_dtype=torch.float32).double() * dY.double()).sum())  # noqa: E731
    for which in range(2):
        W = (Bg, Bu)[which]
        V = torch.where(torch.rand(W.shape, device="cuda") < 0.5, -1.0, 1.0).half()
        up, dn = (W + h * V), (W - h * V)
        V64 = (up.double() - dn.double()) / (2 * h)   # the step as the rounded operands took it
        d = (f(up, Bu) - f(dn, Bu)) if which == 0 else (f(Bg, up) - f(Bg, dn))
        want = float(((g.dBg, g.dBu)[which].double() * V64).sum())
        # The sum has K N terms of random sign: its size is about
        # |dW|_2, to which the errors compare: dZ's and Z's half steps 2^-11
        # each (times the up to 3-fold sensitivity), and third-order terms
        # h^2 / 6 |x.v|^2-ish: (h sqrt K)^2 / 6 = 0.23 % times the same.
        scale = float((g.dBg, g.dBu)[which].double().norm())
        assert abs(d / (2 * h) - want) <= 0.02 * scale, (which, d / (2 * h), want, scale)


def test_training_step_with_clipping():
    torch.manual_seed(2)
    m = mk.GatedFFN(96, 200, bias=True)
    mlp = mk.FusedMLPSoftplus(D=96, H=64, out_features=32, layers=3)
    x = torch.randn(150, 96, device="cuda", dtype=torch.bfloat16)
    mlp(m(x).half()).float().square().sum().backward()
    grads = [p.grad for p in list(m.parameters()) + list(mlp.parameters())]
    want = torch.cat([g.double().flatten() for g in grads]).norm()
    before = [g.double().clone() for g in grads]
    n = mk.clip_grad_norm(grads, 0.5)
    assert abs(float(n) / float(want) - 1) < 1e-6 and float(want) > 0.5
    c = 0.5 / (float(want) + 1e-6)
    for g, b in zip(grads, before):
        assert bool(((g.double() - c * b).abs() <= 2.0 ** -22 * (c * b).abs() + ref.half_step(c * b, g.dtype)).all())


def _state(seed, M=70, D=72, H=136):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to("cuda")  # noqa: E731
    s = dict(x=r(M, D), Wg=r(D, H) / 8, Wu=r(D, H) / 8, Wd=r(H, D) / 12, dy=r(M, D))
    e = lambda *sh, dt=torch.bfloat16: torch.empty(*sh, dtype=dt, device="cuda")  # noqa: E731
    s.update(h=e(M, H), zg=e(M, H), zu=e(M, H), y=e(M, D), dh=e(M, H), dx=e(M, D), dWd=e(H, D), dWg=e(D, H), dWu=e(D, H),
             norm=e((), dt=torch.float32))
    big = max(mk.load_library().coalesce_gated_gemm_backward_workspace_size(M, H, D),
              mk.load_library().coalesce_gemm_residual_backward_workspace_size(M, D, H),
              mk.load_library().coalesce_gated_gemm_workspace_size(M, H, D),
              mk.load_library().coalesce_gemm_residual_workspace_size(M, D, H), 1 << 20)
    s["ws"] = torch.empty(big, dtype=torch.uint8, device="cuda")
    return s


OUTS = ("h", "zg", "zu", "y", "dh", "dx", "dWd", "dWg", "dWu", "norm")


def _step(s, stream=None):
    w = s["ws"]
    mk.gated_gemm_train(s["x"], s["Wg"], s["Wu"], out=s["h"], preact=(s["zg"], s["zu"]), workspace=w, stream=stream)
    mk.gemm_residual(s["h"], s["Wd"], s["x"], out=s["y"], workspace=w, stream=stream)
    mk.gemm_residual_backward(s["h"], s["Wd"], s["dy"], grad_dtype=torch.bfloat16, dA=s["dh"], dB=s["dWd"], workspace=w,
                              stream=stream)
    mk.gated_gemm_backward(s["x"], s["Wg"], s["Wu"], (s["zg"], s["zu"]), s["dh"], grad_dtype=torch.bfloat16, dA=s["dx"],
                           dB=(s["dWg"], s["dWu"]), workspace=w, stream=stream)
    mk.clip_grad_norm([s["dWd"], s["dWg"], s["dWu"]], 1.0, norm=s["norm"], workspace=w, stream=stream)


@pytest.mark.parametrize("M", [3, 70, 700])
def test_graph_replays_match_eager(M):
    s = _state(3, M=M)
    _step(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _step(s)
    gen = torch.Generator().manual_seed(9)
    for rep in range(4):
        for k in ("x", "dy"):
            s[k].copy_(torch.randn(s[k].shape, generator=gen).to(torch.bfloat16))
        _step(s)
        torch.cuda.synchronize()
        want = {k: s[k].clone() for k in OUTS}
        for k in OUTS:
            s[k].fill_(float("nan"))
        s["ws"].fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        for k in OUTS:
            assert torch.equal(s[k], want[k]), "replay %d: %s" % (rep, k)


def test_on_another_stream():
    s = _state(4)
    _step(s)
    torch.cuda.synchronize()
    want = {k: s[k].clone() for k in OUTS}
    for k in OUTS:
        s[k].fill_(float("nan"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    _step(s, stream=side)
    g = mk.gated_gemm_backward(s["x"], s["Wg"], s["Wu"], (s["zg"], s["zu"]), s["dh"], grad_dtype=torch.bfloat16,
                               stream=side)  # outputs and workspace made by the call
    side.synchronize()
    for k in OUTS:
        assert torch.equal(s[k], want[k]), k
    assert torch.equal(g.dA, want["dx"])


def test_backward_captured_while_eager_gradients_live():
    # parameters that have eager gradients and an eager graph alive, then a
    # capture of the whole step on fresh tensors
    torch.manual_seed(5)
    m = mk.GatedFFN(64, 128)
    x = torch.randn(40, 64, device="cuda", dtype=torch.bfloat16)
    keep = m(x)                       # an eager autograd graph of the same leaves stays alive
    torch.autograd.grad(m(x).float().sum(), list(m.parameters()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s = _state(6, M=40, D=64, H=128)
        _step(s)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    want = {k: s[k].clone() for k in OUTS}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _step(s)
    for k in OUTS:
        s[k].zero_()
    graph.replay()
    torch.cuda.synchronize()
    for k in OUTS:
        assert torch.equal(s[k], want[k]), k
    keep.float().sum().backward()
    assert m.Wg.grad is not None
