"""The block with 8-bit weights inside a model that changes its type or device: scales,
biases and norm stay float32, x and the result change."""
import copy

import pytest
import torch

import mlp_megakernel_amd as mk

pytestmark = pytest.mark.gpu

F32 = ("Wg_scale", "Wu_scale", "Wd_scale", "bg", "bu", "bd", "norm_weight", "norm_bias")


def block(dtype=torch.bfloat16):
    torch.manual_seed(3)
    m = mk.GatedFFN(72, 200, bias=True, norm=True, dtype=dtype)
    for b in (m.bg, m.bu, m.bd, m.norm_bias):
        torch.nn.init.normal_(b, std=0.3)
    return m.quantized()


@pytest.mark.parametrize("change,dtype", [
    (lambda m: m.half(), torch.float16), (lambda m: m.bfloat16(), torch.bfloat16), (lambda m: m.float(), torch.float32),
    (lambda m: m.to(torch.float16), torch.float16), (lambda m: m.to("cpu", torch.float16).cuda(), torch.float16),
    (lambda m: m.cpu().to("cuda"), torch.bfloat16), (lambda m: m.half().bfloat16(), torch.bfloat16),
    (lambda m: torch.nn.Sequential(m).half()[0], torch.float16)])
def test_a_change_of_type_is_that_of_x(change, dtype):
    q = block()
    before = {k: v.clone() for k, v in q.state_dict().items()}
    r = change(copy.deepcopy(q))
    assert r.dtype is dtype
    for k, v in r.state_dict().items():
        assert v.is_cuda and v.dtype is before[k].dtype and torch.equal(v, before[k]), k
    assert all(getattr(r, k).dtype is torch.float32 for k in F32)
    # values that every type holds: the results differ by their own rounding, and by the integers of h and of
    # the norm's result, which are quantised from 16 bits or 32 (a step each of their largest magnitudes / 127)
    x = torch.randint(-8, 9, (20, 72), device="cuda").to(torch.bfloat16)
    y, want = r(x.to(dtype)), q(x)
    assert y.dtype is dtype and y.shape == x.shape
    if dtype is torch.bfloat16:
        assert torch.equal(y, want)
    f = (want - x).double()
    assert float(((y.double() - x.double()) - f).norm() / f.norm()) <= 4 * 0.012 + 0.01
    with pytest.raises(ValueError):
        r(x.to(torch.float32 if dtype is not torch.float32 else torch.float16))


@pytest.mark.parametrize("change", [lambda m: m.double(), lambda m: m.type(torch.float16), lambda m: m.to(torch.complex64)])
def test_other_types_are_refused_and_change_nothing(change):
    q = block()
    x = torch.randn(5, 72, device="cuda").bfloat16()
    want = q(x)
    with pytest.raises(TypeError):
        change(q)
    assert torch.equal(q(x), want)


def test_storage_shared_between_processes_and_left_empty():
    q = block()
    cpu = copy.deepcopy(q).cpu().share_memory()
    assert cpu.Wg.is_shared() and cpu.dtype is q.dtype
    x = torch.randn(5, 72, device="cuda").bfloat16()
    assert torch.equal(cpu.cuda()(x), q(x))
    empty = copy.deepcopy(q).to_empty(device="cuda")
    empty.load_state_dict(q.state_dict())
    assert torch.equal(empty(x), q(x))
