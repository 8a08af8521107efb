"""Layer norm, dropout, quantisation and the 8-bit products on a stream of their own
while the current stream still uses memory that was just freed there, and the
blocks made of them over a batch without rows."""
import pytest
import torch

import mlp_megakernel_amd as mk
from helpers import progress
from test_streams_gpu import _beside, _tensors

pytestmark = pytest.mark.gpu

M, N, K = 500, 1032, 4104     # splits its contraction: results and workspace


def _calls():
    gen = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    x, res, dy, w, b = r(M, K), r(M, K), r(M, K), r(K), r(K)
    q, s = mk.quantize_rows(x)
    (bg, sg), (bu, su) = (mk.quantize_columns(r(K, N)) for _ in range(2))
    y, total, stats = mk.add_layer_norm_train(x, res, w, b, p=0.25, seed=3)
    return {
        "layer_norm": lambda st: mk.layer_norm_train(x, w, b, stream=st),
        "add_layer_norm": lambda st: mk.add_layer_norm_train(x, res, w, b, p=0.25, seed=3, stream=st),
        "layer_norm_backward": lambda st: mk.layer_norm_backward(total, w, stats, dy, p=0.25, seed=3,
                                                                 want_dbranch=True, stream=st),
        "dropout": lambda st: mk.dropout(x, 0.25, 3, stream=st),
        "dropout_backward": lambda st: mk.dropout_backward(dy, 0.25, 3, stream=st),
        "quantize_rows": lambda st: mk.quantize_rows(x, stream=st),
        "quantize_columns": lambda st: mk.quantize_columns(x, stream=st),
        "gemm_int8": lambda st: mk.gemm_int8(q, bg, s, sg, stream=st),
        "gated_gemm_int8": lambda st: mk.gated_gemm_int8(q, bg, bu, s, sg, su, stream=st),
    }


@pytest.mark.parametrize("name", ["layer_norm", "add_layer_norm", "layer_norm_backward", "dropout", "dropout_backward",
                                  "quantize_rows", "quantize_columns", "gemm_int8", "gated_gemm_int8"])
def test_memory_freed_on_the_current_stream_is_not_taken(name):
    call = _calls()[name]
    want = _tensors(call(None))
    _beside(call, want, torch.cuda.Stream())
    progress(name)


@pytest.mark.parametrize("shape", [(0, 64), (2, 0, 64)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_a_batch_without_rows(shape, dtype):
    layer = mk.GatedFFN(64, 160, bias=True, norm=True, dropout=0.25).to("cuda", dtype)
    x = torch.zeros(*shape, device="cuda", dtype=dtype, requires_grad=True)
    y = layer(x)
    assert y.shape == x.shape and y.dtype == dtype
    y.sum().backward()
    assert x.grad.shape == x.shape
    for name, q in layer.named_parameters():
        assert q.grad is not None and not bool(q.grad.any()), name
    assert layer.eval().quantized()(x.detach()).shape == x.shape
