"""GatedFFN called in ways that its kernels do not serve: each is refused, and
what stands next to it still works."""
import pytest
import torch
import torch.autograd.forward_ad as fw

import mlp_megakernel_amd as mk

pytestmark = pytest.mark.gpu


def _module(**kw):
    torch.manual_seed(0)
    m = mk.GatedFFN(64, 128, **kw)
    return m, torch.randn(8, 64, device="cuda", dtype=torch.bfloat16)


@pytest.mark.parametrize("frozen", [False, True])
def test_forward_mode_is_refused(frozen):
    m, x = _module()
    want = m(x).detach()
    m.requires_grad_(not frozen)
    v = torch.ones_like(x)
    with fw.dual_level():
        with torch.set_grad_enabled(frozen):      # frozen parameters, or no_grad: the call without autograd
            with pytest.raises(NotImplementedError):
                m(fw.make_dual(x, v))
            assert torch.equal(m(x), want)
        # a parameter that carries a tangent
        p = {k: t.detach() for k, t in m.named_parameters()}
        p["Wd"] = fw.make_dual(p["Wd"], torch.ones_like(p["Wd"]))
        with pytest.raises(NotImplementedError):
            torch.func.functional_call(m, p, (x,))


def test_trace_without_gradients_is_refused():
    m, x = _module()
    with torch.no_grad(), pytest.raises(RuntimeError, match="traced"):
        torch.jit.trace(m, (x,), check_trace=False)
    m.requires_grad_(False)
    with pytest.raises(RuntimeError, match="traced"):
        torch.jit.trace(m, (x,), check_trace=False)
    m.requires_grad_(True)
    t = torch.jit.trace(m, (x,), check_trace=False)
    y = torch.randn_like(x)
    assert torch.equal(t(y), m(y))


@pytest.mark.parametrize("shape", [(4, 32), (2, 128), (64, 1), (32,), (2, 2, 32)])
def test_inputs_of_another_width_are_refused(shape):
    # 64 elements each row, or a multiple: they would fill rows of the right width
    m, _ = _module()
    x = torch.randn(shape, device="cuda", dtype=torch.bfloat16)
    for grad in (False, True):
        with torch.set_grad_enabled(grad), pytest.raises(ValueError, match="64"):
            m(x)
    for good in ((64,), (0, 64), (3, 1, 64), (2, 0, 64)):
        assert m(torch.zeros(good, device="cuda", dtype=torch.bfloat16)).shape == good
    with pytest.raises(ValueError):
        m(torch.zeros((), device="cuda", dtype=torch.bfloat16))


@pytest.mark.parametrize("D,H", [(72, 128), (71, 130)])
def test_parameters_in_one_flat_buffer(D, H):
    # as an optimizer's or a checkpoint's flat buffer holds them: only element alignment
    torch.manual_seed(1)
    m, plain = (mk.GatedFFN(D, H, bias=True) for _ in range(2))
    flat = torch.zeros(sum(p.numel() for p in m.parameters()) + 3, device="cuda", dtype=torch.bfloat16)
    at = 3
    for p, q in zip(m.parameters(), plain.parameters()):
        q.data.normal_(std=0.1)
        part = flat[at:at + p.numel()].view(p.shape)
        part.copy_(q.data)
        p.data = part
        at += p.numel()
    assert any(p.data_ptr() % 16 for p in (m.bg, m.bu, m.bd))
    x = torch.randn(20, D, device="cuda", dtype=torch.bfloat16)
    a, b = m(x), plain(x)
    a.backward(x)
    b.backward(x)
    assert torch.equal(a, b)
    for p, q in zip(m.parameters(), plain.parameters()):
        assert torch.equal(p.grad, q.grad)
    with torch.no_grad():
        assert torch.equal(m(x), a)


def test_training_forms_check_their_arguments():
    A, B = (torch.zeros(s, device="cuda", dtype=torch.bfloat16) for s in ((8, 64), (64, 32)))
    for bad in (B[0], B[None], B.cpu(), B.float(), B[:32]):
        for call in (lambda: mk.gemm_residual_train(A, bad), lambda: mk.gated_gemm_train(A, bad, bad)):
            with pytest.raises(ValueError):
                call()
    for bad in (A[0], A[None], A.cpu(), A.float()):
        for call in (lambda: mk.gemm_residual_train(bad, B), lambda: mk.gated_gemm_train(bad, B, B)):
            with pytest.raises(ValueError):
                call()
