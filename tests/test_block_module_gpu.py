"""The block as a whole, with its norm and dropout and in 8 bits: values and every
gradient against fp64 under the mask that was drawn, against differences, captured
and replayed, moved and stored."""
import copy
import io

import pytest
import torch

import block_reference as ref
import ffn_reference as fref
import mlp_megakernel_amd as mk
import mlp_megakernel_amd.ffn as ffn
from ffn_reference import U32 as U

pytestmark = pytest.mark.gpu


def block64(p, x, act, residual, eps, keep, scale):
    n = x
    if "norm_weight" in p:
        d = x - x.mean(-1, keepdim=True)
        n = d / torch.sqrt(d.square().mean(-1, keepdim=True) + eps) * p["norm_weight"] + p["norm_bias"]
    zg, zu = n @ p["Wg"], n @ p["Wu"]
    if "bg" in p:
        zg, zu = zg + p["bg"], zu + p["bu"]
    y = (fref.act(zg, act) * zu) @ p["Wd"]
    if "bd" in p:
        y = y + p["bd"]
    if keep is not None:
        y = y * keep * scale
    return x + y if residual else y


def rel(a, b):
    return float((a.to(torch.float64) - b).norm() / b.norm())


def fixed_seed(monkeypatch, seed=77, offset=5):
    both = torch.tensor([seed, offset], device="cuda")
    monkeypatch.setattr(ffn, "_draw_seed", lambda device: both)
    return both


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("act,bias,residual,norm,p,shape", [
    ("silu", False, True, True, 0.0, (3, 17, 64)), ("gelu", True, True, True, 0.2, (130, 72)),
    ("silu", True, False, True, 0.5, (1, 100)), ("relu", True, True, False, 0.25, (2, 33, 71)),
    ("silu", False, False, False, 0.1, (40, 96)), ("gelu", True, True, True, 0.3, (9, 71))])
def test_block_matches_fp64(monkeypatch, dt, act, bias, residual, norm, p, shape):
    torch.manual_seed(0)
    fixed_seed(monkeypatch)
    D, H = shape[-1], 2 * shape[-1] + 37
    m = mk.GatedFFN(D, H, act=act, bias=bias, residual=residual, dtype=dt, norm=norm, dropout=p)
    for b in ([m.bg, m.bu, m.bd] if bias else []) + ([m.norm_bias] if norm else []):
        torch.nn.init.normal_(b, std=0.3)
    if norm:
        torch.nn.init.normal_(m.norm_weight, 1.0, 0.2)
    x = (torch.randn(shape, device="cuda") * 1.5 + 0.25).to(dt).requires_grad_()
    dy = torch.randn(shape, device="cuda").to(dt)
    y = m(x)
    y.backward(dy)
    with torch.no_grad():
        assert torch.equal(m(x), y), "inference and training forward differ"
    q = {k: v.detach().to(torch.float64).requires_grad_() for k, v in m.named_parameters()}
    x64 = x.detach().to(torch.float64).requires_grad_()
    rows = x.numel() // D
    keep = ref.kept(rows, D, p, 77, 5).reshape(shape).to(torch.float64) if p else None
    y64 = block64(q, x64, act, residual, 1e-5, keep, 1 / (1 - p))
    y64.backward(dy.to(torch.float64))
    # Roundings to the type between the inputs and any gradient: n, Z, H or dH, the
    # dropped dY, dZ, dn, the output: 7, each at most half a step relative to its
    # operands, which stay within a factor 4 of the result in norm here.
    tol = 7 * 4 * torch.finfo(dt).eps / 2
    assert rel(y, y64) <= tol
    assert rel(x.grad, x64.grad) <= tol
    for k, v in m.named_parameters():
        assert v.grad is not None and v.grad.dtype == dt and rel(v.grad, q[k].grad) <= tol, k


def test_gradient_of_the_norm_against_differences():
    # <dY, f(w + h v) - f(w - h v)> / 2h against <dw, v>: h = 1/8 in bf16 is exact for w = 1;
    # f is close to linear in w (silu's curvature: h^2 / 6 of third derivatives, below 1 %),
    # and each f is rounded by 2^-9 of its size, which the 4000 terms average out
    torch.manual_seed(1)
    m = mk.GatedFFN(64, 160, norm=True, residual=False)
    x, dy = torch.randn(200, 64, device="cuda").bfloat16(), torch.randn(200, 64, device="cuda").bfloat16()
    v = torch.randint(0, 2, (64,), device="cuda").bfloat16() * 2 - 1
    m(x).backward(dy)
    want = float((m.norm_weight.grad.double() * v.double()).sum())

    def f(s):
        with torch.no_grad():
            m.norm_weight.copy_(1 + s * v)
            return float((m(x).double() * dy.double()).sum())

    h = 0.125
    scale = float(m.norm_weight.grad.double().norm()) * 8  # of <dw, v>, v of 64 signs
    assert abs((f(h) - f(-h)) / (2 * h) - want) <= 0.1 * scale


def test_dropout_goes_by_torchs_generator():
    m = mk.GatedFFN(64, 128, dropout=0.5, residual=False)
    x = torch.randn(30, 64, device="cuda").bfloat16()
    torch.manual_seed(3)
    a, b = m(x), m(x)
    torch.manual_seed(3)
    assert torch.equal(m(x), a) and not torch.equal(a, b)
    share = float((a == 0).float().mean())
    assert abs(share - 0.5) <= 5 * (0.25 / a.numel()) ** 0.5 + 0.01  # (products that are 0 by themselves)
    m.eval()
    assert torch.equal(m(x), m(x)) and not bool((m(x) == 0).any())
    # recomputed in the backward, as a checkpoint does, the mask is the same
    m.train()
    from torch.utils.checkpoint import checkpoint
    x1, x2 = (x.clone().requires_grad_() for _ in range(2))
    torch.manual_seed(4)
    m(x1).float().sum().backward()
    torch.manual_seed(4)
    checkpoint(m, x2, use_reentrant=False).float().sum().backward()
    assert torch.equal(x1.grad, x2.grad)


def test_captured_training_step(monkeypatch):
    torch.manual_seed(5)
    m = mk.GatedFFN(72, 200, norm=True, dropout=0.25, bias=True)
    x = torch.randn(50, 72, device="cuda").bfloat16()
    params = list(m.parameters())

    def step():
        y = m(x)
        return (y, *torch.autograd.grad(y.float().square().sum(), params))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    # with torch's generator every replay has a mask of its own
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        held = step()
    seen = []
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        seen.append(held[0].clone())
    assert not torch.equal(seen[0], seen[1]) and not torch.equal(seen[1], seen[2])
    # with a seed that stays, it is the eager step's
    both = fixed_seed(monkeypatch)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        held = step()
    for i in range(4):
        both.copy_(torch.tensor([i, 9]))
        x.add_(0.125)
        with torch.cuda.stream(side):
            want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))


def test_only_what_is_wanted():
    torch.manual_seed(6)
    m = mk.GatedFFN(64, 128, norm=True)
    x = torch.randn(20, 64, device="cuda").bfloat16()
    m(x).float().sum().backward()
    full = {k: v.grad.clone() for k, v in m.named_parameters()}
    for name in ("norm_weight", "norm_bias", "Wd", "Wg"):
        m.zero_grad()
        for k, v in m.named_parameters():
            v.requires_grad_(k == name)
        m(x).float().sum().backward()
        for k, v in m.named_parameters():
            assert (v.grad is not None) == (k == name)
        assert torch.equal(getattr(m, name).grad, full[name])


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("act,bias,residual,norm,D,H", [
    ("silu", False, True, False, 64, 160), ("gelu", True, True, True, 71, 203), ("relu", True, False, True, 136, 328)])
def test_quantized_block(dt, act, bias, residual, norm, D, H):
    torch.manual_seed(7)
    m = mk.GatedFFN(D, H, act=act, bias=bias, residual=residual, dtype=dt, norm=norm)
    for b in ([m.bg, m.bu, m.bd] if bias else []) + ([m.norm_bias] if norm else []):
        torch.nn.init.normal_(b, std=0.3)
    x = torch.randn(3, 31, D, device="cuda").to(dt)
    q = m.quantized()
    with torch.no_grad():
        y, y16 = q(x), m(x)
    x2 = mk.aligned_copy(x.reshape(-1, D))
    n = mk.layer_norm(x2, m.norm_weight.float(), m.norm_bias.float(), out_dtype=dt) if norm else x2
    back = lambda t: ref.f64(t[0]) * ref.f64(t[1])[:, None]  # noqa: E731
    X = back(mk.quantize_rows(mk.aligned_copy(n)))
    W = {k: back((getattr(q, k), getattr(q, k + "_scale"))).t() for k in ("Wg", "Wu", "Wd")}
    for k in W:  # the weights: half a step of their channel
        w = ref.f64(getattr(m, k))
        assert bool(((W[k] - w).abs() <= 0.501 * ref.f64(getattr(q, k + "_scale"))[None, :]).all())
    b64 = lambda b: ref.f64(b) if b is not None else 0.0  # noqa: E731
    zg, zu = X @ W["Wg"] + b64(m.bg), X @ W["Wu"] + b64(m.bu)
    # z is known to 3 roundings of fp32 from exact sums; scales are as stored
    ez = lambda z: 4 * U * (z.abs() + 1)  # noqa: E731
    f, ef = fref.act_bound(zg, ez(zg), act, False)
    h = f * zu
    eh = fref.rounded(h, f.abs() * ez(zu) + zu.abs() * ef + U * h.abs(), dt)
    # h is quantised in steps of its row's largest magnitude / 127
    step = (h.abs() + eh).amax(1, keepdim=True) / 127
    e = (0.501 * step + eh) @ W["Wd"].abs()
    v = h @ W["Wd"] + b64(m.bd)
    e = e + 4 * U * (v.abs() + e)
    if residual:
        v = v + ref.f64(x2)
        e = e + U * (v.abs() + e)
    ref.check(y.reshape(-1, D), (v, fref.rounded(v, e, dt)), "y")
    # and it is near the block it was made of: two quantisations of both operands, each
    # a step of amax / 127 (amax below 5 deviations) / sqrt(12), 1.2 % each, over two products
    base = x if residual else torch.zeros_like(x)
    assert rel((y - base).float(), (y16.double() - base.double())) <= 4 * 0.012 + 0.01


def test_quantized_tokens_do_not_depend_on_each_other():
    torch.manual_seed(8)
    q = mk.GatedFFN(200, 520, norm=True, bias=True).quantized()
    x = torch.randn(300, 200, device="cuda").bfloat16()
    with torch.no_grad():
        y = q(x)
        for a, b in ((0, 1), (7, 9), (20, 80), (100, 299)):
            assert torch.equal(q(x[a:b]), y[a:b])
        assert q(x[:0]).shape == (0, 200)


@pytest.mark.parametrize("D,H", [(64, 160), (70, 203)])
def test_quantized_block_is_stored_moved_and_captured(D, H):
    torch.manual_seed(9)
    m = mk.GatedFFN(D, H, norm=True, bias=True)
    q = m.quantized()
    x = torch.randn(5, D, device="cuda").bfloat16()
    want = q(x)
    f = io.BytesIO()
    torch.save(q.state_dict(), f)
    f.seek(0)
    other = mk.GatedFFN(D, H, norm=True, bias=True).quantized()
    other.load_state_dict(torch.load(f, weights_only=True))
    for r in (other, copy.deepcopy(q), copy.deepcopy(q).cpu().cuda()):
        assert torch.equal(r(x), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        held = q(x)
    for _ in range(3):
        x.mul_(1.5)
        want = q(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, want)


def test_refusals():
    x = torch.randn(4, 64, device="cuda").bfloat16()
    m = mk.GatedFFN(64, 128, norm=True, dropout=0.1)
    q = m.quantized()
    with pytest.raises(ValueError):
        mk.GatedFFN(64, 128, dropout=1.5)
    for bad in (x[:, :32], x.half(), x.float()):
        with pytest.raises(ValueError):
            q(bad)
    with pytest.raises(RuntimeError):
        q(x.clone().requires_grad_())
    with torch.no_grad():
        assert q(x.clone().requires_grad_()).shape == x.shape
        with pytest.raises(RuntimeError):
            torch.jit.trace(q, x)
        with pytest.raises(RuntimeError):
            torch.jit.trace(m, x)
    with torch.autograd.forward_ad.dual_level():
        dual = torch.autograd.forward_ad.make_dual(x, torch.ones_like(x))
        with torch.no_grad(), pytest.raises(NotImplementedError):
            q(dual)


def test_a_block_stored_without_norm_and_dropout():
    # modules pickled before those existed lack the attributes
    m = mk.GatedFFN(64, 128)
    state = {k: v for k, v in m.__dict__.items() if k not in ("norm", "dropout", "eps", "norm_weight", "norm_bias")}
    old = mk.GatedFFN.__new__(mk.GatedFFN)
    old.__setstate__(state)
    x = torch.randn(4, 64, device="cuda").bfloat16()
    with torch.no_grad():
        assert torch.equal(old(x), m(x))
    assert sorted(m.state_dict()) == ["Wd", "Wg", "Wu"]


def test_quantized_block_with_its_vectors_in_a_flat_buffer():
    # as load_state_dict(assign=True) may leave them: at any multiple of 4 bytes
    torch.manual_seed(4)
    block = mk.GatedFFN(64, 160, bias=True, norm=True).quantized()
    x = torch.randn(5, 64, device="cuda", dtype=torch.bfloat16)
    want = block(x)
    vectors = {n: b for n, b in block.named_buffers() if b.dim() == 1}
    flat, at = torch.empty(sum(b.numel() for b in vectors.values()) + 1, device="cuda"), 1
    for n, b in vectors.items():
        part = flat[at:at + b.numel()]
        part.copy_(b)
        setattr(block, n, part)
        at += b.numel()
    assert len(vectors) == 8 and torch.equal(block(x), want)
