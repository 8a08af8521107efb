"""Calls on a stream of their own while the current stream still uses memory
that was just freed there: what a call makes must not lie in it."""
import pytest
import torch

import mlp_megakernel_amd as mk
from helpers import progress

pytestmark = pytest.mark.gpu

M, N, K = 500, 1032, 4104     # splits its contraction: results and workspace


def _inputs():
    gen = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=torch.bfloat16) * K ** -0.25  # noqa: E731
    return r(M, K), r(K, N), r(K, N), r(M, N), r(M, N)


def _tensors(r):
    return [t for v in r for t in _tensors(v)] if isinstance(r, (tuple, list)) else [r]


def _calls(A, Bg, Bu, R, dY):
    Z = mk.gated_gemm_train(A, Bg, Bu)[1]
    grads = [R.clone(), dY.clone()]
    return {
        "gated_gemm": lambda s: mk.gated_gemm(A, Bg, Bu, stream=s),
        "gated_gemm_train": lambda s: mk.gated_gemm_train(A, Bg, Bu, stream=s),
        "gemm_residual": lambda s: mk.gemm_residual(A, Bg, R, stream=s),
        "gemm_residual_train": lambda s: mk.gemm_residual_train(A, Bg, R, act="gelu", stream=s),
        "gated_gemm_backward": lambda s: mk.gated_gemm_backward(A, Bg, Bu, Z, dY, want_dbias=True, stream=s),
        "gemm_residual_backward": lambda s: mk.gemm_residual_backward(A, Bg, dY, Z[0], act="gelu", want_dbias=True,
                                                                      stream=s),
        "grad_norm": lambda s: mk.grad_norm(grads, stream=s),
    }


NAMES = ["gated_gemm", "gated_gemm_train", "gemm_residual", "gemm_residual_train", "gated_gemm_backward",
         "gemm_residual_backward", "grad_norm"]


def _beside(call, want, side):
    """The call on `side` while the current stream, busy for some milliseconds, has yet to read blocks of every size
    that were freed there."""
    sizes = sorted({t.untyped_storage().nbytes() for t in want} | {1 << p for p in range(9, 27)})
    torch.cuda.synchronize()
    held = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
    blocks = [(t.data_ptr(), t.data_ptr() + t.numel()) for t in held]
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(20_000_000)
    read = [(t != 7).sum() for t in held]
    del held
    got = _tensors(call(side))
    for t in got:
        lo = t.untyped_storage().data_ptr()
        assert all(lo + t.untyped_storage().nbytes() <= a or lo >= b for a, b in blocks), "a block still in use"
    side.synchronize()
    torch.cuda.synchronize()
    assert sum(int(n) for n in read) == 0, "memory of the current stream was written"
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", NAMES)
def test_memory_freed_on_the_current_stream_is_not_taken(name):
    call = _calls(*_inputs())[name]
    want = _tensors(call(None))
    _beside(call, want, torch.cuda.Stream())
    progress(name)


@pytest.mark.parametrize("handle", [lambda s: s, lambda s: s.cuda_stream], ids=["stream", "handle"])
def test_result_used_and_freed_on_the_current_stream(handle):
    # the result's block goes back to the side stream's pool only once the
    # current stream, which copies it late, is done with it
    A, Bg, Bu, R, _ = _inputs()
    want = mk.gated_gemm(A, Bg, Bu)
    side, cur = torch.cuda.Stream(), torch.cuda.current_stream()
    side.wait_stream(cur)
    H = mk.gated_gemm(A, Bg, Bu, stream=handle(side))
    cur.wait_stream(side)
    torch.cuda._sleep(20_000_000)
    copy = H.clone()
    del H
    others = [mk.gemm_residual(A, Bg, R, stream=handle(side)) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(copy, want) and all(torch.equal(o, others[0]) for o in others)


def test_default_stream_by_its_handle():
    A, Bg, Bu, _, _ = _inputs()
    assert torch.equal(mk.gated_gemm(A, Bg, Bu, stream=0), mk.gated_gemm(A, Bg, Bu))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        H = mk.gated_gemm(A, Bg, Bu, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(H, mk.gated_gemm(A, Bg, Bu))


def _chain():
    gen = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").half()  # noqa: E731
    x, Ws, dy = r(3000, 128), [r(128, 128) / 16 for _ in range(3)], r(3000, 128)
    acts = mk.mlp_forward_train(x, Ws)[1]
    g = [r(128).abs() for _ in Ws]
    X, b = r(700, 136), r(136)
    f32 = [w.float() for w in Ws]
    return {
        "gemm_bias_act": lambda s: mk.gemm_bias_act(x, Ws[0], g[0], stream=s),
        "mlp_forward": lambda s: mk.mlp_forward(x, Ws, stream=s),
        "mlp_forward_train": lambda s: mk.mlp_forward_train(x, Ws, stream=s),
        "mlp_backward": lambda s: mk.mlp_backward(x, Ws, acts, dy, stream=s),
        "weight_norm": lambda s: mk.weight_norm(Ws, g, stream=s),
        "weight_norm_backward": lambda s: mk.weight_norm_backward(Ws, g, f32, stream=s),
        "bias_add": lambda s: mk.bias_add(X, b, stream=s),
        "activation": lambda s: mk.activation(X, stream=s),
    }


CHAIN = ["gemm_bias_act", "mlp_forward", "mlp_forward_train", "mlp_backward", "weight_norm", "weight_norm_backward",
         "bias_add", "activation"]


@pytest.mark.parametrize("name", CHAIN)
def test_other_entry_points_take_no_memory_in_use(name):
    call = _chain()[name]
    _beside(call, _tensors(call(None)), torch.cuda.Stream())
    progress(name)
