"""The feed-forward products on 8-bit operands, and the quantisation that makes them.

As the rest of the binding: argument checks and marshalling only, all
arithmetic in ``libcoalesce.so``.  Tensors must live on one device; the calls
run there, on ``stream`` or that device's current stream.  They have no gradients.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import _DTYPES, _check, _empty, _matrix, _ptr, load_library
from .ffn import (_act, _current_device, _mat, _new, _one_pitch, _raw_stream, _row_pitch, _short, _there, _vec,
                  _workspace)


def _int8_pitch(cols: int) -> int:
    """A row of bytes up to the next multiple of 16."""
    return max(16, (cols + 15) & -16)


def _new_int8(rows: int, cols: int, device, stream):
    ld = _int8_pitch(cols)
    t = _empty((rows, ld), torch.int8, device, stream)
    return t if ld == cols else t[:, :cols]


def _mat8(t: torch.Tensor, name: str, rows: int, cols: int, dev: int) -> int:
    """The pitch of a rows x cols operand of 8-bit integers (a single row has none)."""
    ld = _mat(t, name, rows, cols, torch.int8, dev)
    return ld if rows > 1 else _int8_pitch(cols)


def quantize_rows(x: torch.Tensor, out: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                  stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(q, scale): the rows of ``x`` as 8-bit integers, x = q * scale[:, None] up to
    half a step, scale = largest magnitude / 127 in float32 (coalesce_quantize_rows).

    A row that holds an infinity or a NaN has scale NaN.
    """
    return _quantize(x, out, scale, stream, False)


def quantize_columns(x: torch.Tensor, out: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                     stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(q, scale): the columns of ``x`` as rows of 8-bit integers, x = (q *
    scale[:, None]).t() up to half a step (coalesce_quantize_columns): what makes
    the weights of :func:`gemm_int8` from those of :func:`gemm_residual`."""
    return _quantize(x, out, scale, stream, True)


def _quantize(x, out, scale, stream, columns):
    if x.is_cuda and x.dim() == 2:
        rows, cols = x.shape[::-1] if columns else x.shape
        if out is None:
            out = _new_int8(rows, cols, x.device, stream)
        if scale is None:
            scale = _empty(rows, torch.float32, x.device, stream)
        status = _short("quantize", "coalesce_quantize_columns" if columns else "coalesce_quantize_rows", stream,
                        columns, x, out, scale)
        if status == 0:
            return out, scale
        if status is not None:
            _check(status)
    M, N, ldx = _matrix(x, "x")
    dev = x.get_device()
    if x.dtype not in _DTYPES:
        raise ValueError("x must be float32, float16 or bfloat16")
    if _current_device() != dev:
        return _there(dev, _quantize, x, out, scale, stream, columns)
    rows, cols = (N, M) if columns else (M, N)
    ldq = _mat8(out, "out", rows, cols, dev)
    _vec(scale, "scale", rows, torch.float32, dev)
    call = load_library().coalesce_quantize_columns if columns else load_library().coalesce_quantize_rows
    _check(call(x.data_ptr(), ldx if M > 1 else _row_pitch(N, x.dtype), out.data_ptr(), ldq, scale.data_ptr(), M, N,
                _DTYPES[x.dtype], _raw_stream(stream, dev)))
    return out, scale


def _tokens(A: torch.Tensor):
    M, K, ld = _matrix(A, "A")
    if A.dtype is not torch.int8:
        raise ValueError("A must be int8")
    return M, K, ld if M > 1 else _int8_pitch(K), A.get_device()


def _channels(B: torch.Tensor, name: str) -> int:
    if B.dim() != 2:
        raise ValueError("%s must be 2-D" % name)
    return B.shape[0]


def _out_type(out_dtype, out, residual):
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else residual.dtype if residual is not None else torch.bfloat16
    if out_dtype not in _DTYPES:
        raise ValueError("the result must be float32, float16 or bfloat16")
    return out_dtype


def gemm_int8(A: torch.Tensor, B: torch.Tensor, a_scale: torch.Tensor, b_scale: torch.Tensor,
              bias: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None, act="none",
              out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
              workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Y = act((A @ B.t()) * a_scale[:, None] * b_scale + bias) + residual in one
    fused kernel (coalesce_gemm_int8).

    A is M x K and B N x K, int8 with rows on 16-byte boundaries, K at most 131071;
    the scales (one per row of each) and the bias are float32.  The result is
    float32, float16 or bfloat16 (``out_dtype``, else that of ``out`` or of the
    residual, else bfloat16); the residual has its type and may be ``out``.
    """
    # (what is no pair of matrices is left to the checks below)
    if A.is_cuda and A.dim() == B.dim() == 2 and A.get_device() == _current_device():
        M, K, N = A.shape + B.shape[:1]
        odt = _out_type(out_dtype, out, residual)
        if out is None:
            out = _new(M, N, odt, A.device, stream)
        ws, nws, _keep = _workspace("coalesce_gemm_int8_workspace_size", A.get_device(), M, N, K, workspace, stream)
        status = None
        if out.dtype is odt:
            status = _short("gemm_int8", "coalesce_gemm_int8", stream, A, B, a_scale, b_scale, bias, residual, out,
                            _act(act), ws, nws)
        if status == 0:
            return out
        if status is not None:
            _check(status)
    M, K, lda, dev = _tokens(A)
    if _current_device() != dev:
        return _there(dev, gemm_int8, A, B, a_scale, b_scale, bias, residual, act, out_dtype, out, workspace, stream)
    N = _channels(B, "B")
    ldb = _mat8(B, "B", N, K, dev)
    _vec(a_scale, "a_scale", M, torch.float32, dev)
    _vec(b_scale, "b_scale", N, torch.float32, dev)
    _vec(bias, "bias", N, torch.float32, dev)
    odt, a = _out_type(out_dtype, out, residual), _act(act)
    ldr = 0 if residual is None else _mat(residual, "residual", M, N, odt, dev)
    if out is None:
        out = _new(M, N, odt, A.device, stream)
    ldy = _mat(out, "out", M, N, odt, dev)
    ws, nws, _keep = _workspace("coalesce_gemm_int8_workspace_size", dev, M, N, K, workspace, stream)
    _check(load_library().coalesce_gemm_int8(
        A.data_ptr(), lda, B.data_ptr(), ldb, a_scale.data_ptr(), b_scale.data_ptr(), _ptr(bias), _ptr(residual), ldr,
        out.data_ptr(), ldy, M, N, K, _DTYPES[odt], a, ws, nws, _raw_stream(stream, dev)))
    return out


def gated_gemm_int8(A: torch.Tensor, Bg: torch.Tensor, Bu: torch.Tensor, a_scale: torch.Tensor,
                    bg_scale: torch.Tensor, bu_scale: torch.Tensor, bias_g: Optional[torch.Tensor] = None,
                    bias_u: Optional[torch.Tensor] = None, act="silu", out_dtype: Optional[torch.dtype] = None,
                    out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """act(zg) * zu with z = (A @ B.t()) * a_scale[:, None] * b_scale + bias for both
    weights, in one fused kernel (coalesce_gated_gemm_int8); operands as in
    :func:`gemm_int8`, Bg and Bu of one row pitch."""
    # (what is no pair of matrices is left to the checks below)
    if A.is_cuda and A.dim() == Bg.dim() == 2 and A.get_device() == _current_device():
        M, K, N = A.shape + Bg.shape[:1]
        odt = _out_type(out_dtype, out, None)
        if out is None:
            out = _new(M, N, odt, A.device, stream)
        ws, nws, _keep = _workspace("coalesce_gated_gemm_int8_workspace_size", A.get_device(), M, N, K, workspace, stream)
        status = None
        if out.dtype is odt:
            status = _short("gated_gemm_int8", "coalesce_gated_gemm_int8", stream, A, Bg, Bu, a_scale, bg_scale,
                            bu_scale, bias_g, bias_u, out, _act(act), ws, nws)
        if status == 0:
            return out
        if status is not None:
            _check(status)
    M, K, lda, dev = _tokens(A)
    if _current_device() != dev:
        return _there(dev, gated_gemm_int8, A, Bg, Bu, a_scale, bg_scale, bu_scale, bias_g, bias_u, act, out_dtype, out,
                      workspace, stream)
    N = _channels(Bg, "Bg")
    ldb = _one_pitch((Bg, Bu), ("Bg", "Bu"), N, K, torch.int8, dev) if N > 1 else _mat8(Bg, "Bg", N, K, dev)
    if N <= 1:
        _mat8(Bu, "Bu", N, K, dev)
    _vec(a_scale, "a_scale", M, torch.float32, dev)
    _vec(bg_scale, "bg_scale", N, torch.float32, dev)
    _vec(bu_scale, "bu_scale", N, torch.float32, dev)
    _vec(bias_g, "bias_g", N, torch.float32, dev)
    _vec(bias_u, "bias_u", N, torch.float32, dev)
    odt, a = _out_type(out_dtype, out, None), _act(act)
    if out is None:
        out = _new(M, N, odt, A.device, stream)
    ldy = _mat(out, "out", M, N, odt, dev)
    ws, nws, _keep = _workspace("coalesce_gated_gemm_int8_workspace_size", dev, M, N, K, workspace, stream)
    _check(load_library().coalesce_gated_gemm_int8(
        A.data_ptr(), lda, Bg.data_ptr(), Bu.data_ptr(), ldb, a_scale.data_ptr(), bg_scale.data_ptr(),
        bu_scale.data_ptr(), _ptr(bias_g), _ptr(bias_u), out.data_ptr(), ldy, M, N, K, _DTYPES[odt], a, ws, nws,
        _raw_stream(stream, dev)))
    return out
