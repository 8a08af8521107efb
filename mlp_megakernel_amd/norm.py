"""Layer norm of a residual stream and dropout: what stands between the products of a block.

As the rest of the binding: argument checks and marshalling only, all
arithmetic in ``libcoalesce.so``.  Tensors are 2-D with 16-byte aligned rows (any
number of columns) and live on one device; the calls run there, on ``stream`` or
that device's current stream.  They are not seen by autograd: results have no
gradient, whatever the operands require (:class:`GatedFFN` does).
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple, Optional, Tuple, Union

import torch

from . import _DTYPES, _check, _empty, _matrix, _ptr, _stream_object, load_library
from .ffn import _current_device, _mat, _new, _raw_stream, _row_pitch, _short, _take, _there, _vec, _ws_sizes

Seed = Union[int, torch.Tensor]


class NormGrads(NamedTuple):
    """Gradients of :func:`layer_norm` and :func:`add_layer_norm` (``None``: not wanted)."""
    dx: Optional[torch.Tensor]       # of the stream (and of the residual, which is the stream before the sum)
    dbranch: Optional[torch.Tensor]  # of the branch that add_layer_norm dropped out and added
    dweight: Optional[torch.Tensor]
    dbias: Optional[torch.Tensor]


def _rows(t: torch.Tensor, name: str):
    """(rows, cols, pitch, device) of the operand that the others go by."""
    rows, cols, ld = _matrix(t, name)
    if t.dtype not in _DTYPES:
        raise ValueError("%s must be float32, float16 or bfloat16" % name)
    return rows, cols, ld if rows > 1 else _row_pitch(cols, t.dtype), t.get_device()


def _mask(p: float, seed: Seed, offset: int, dev: int):
    """(p, seed, offset, pointer to both in device memory) of a dropout mask."""
    if isinstance(seed, torch.Tensor):
        if seed.shape != (2,) or seed.dtype is not torch.int64 or not seed.is_contiguous() or seed.get_device() != dev:
            raise ValueError("a seed in device memory must be two contiguous int64 (seed, offset) on GPU %d" % dev)
        if offset:
            raise ValueError("offset stands beside the seed in device memory")
        return float(p), 0, 0, seed.data_ptr()
    return float(p), int(seed) & 0xFFFFFFFFFFFFFFFF, int(offset) & 0xFFFFFFFFFFFFFFFF, None


def _affine(weight, bias, N: int, dtype: torch.dtype, dev: int) -> torch.dtype:
    """Checks weight and bias; the type they share."""
    wt = weight.dtype if weight is not None else bias.dtype if bias is not None else dtype
    if wt is not torch.float32 and wt is not dtype:
        raise ValueError("weight and bias must be float32 or %s" % dtype)
    _vec(weight, "weight", N, wt, dev)
    _vec(bias, "bias", N, wt, dev)
    return wt


def _stats(stats, M: int, dev: int):
    if len(stats) != 2:
        raise ValueError("stats must be (mean, rstd)")
    _vec(stats[0], "mean", M, torch.float32, dev)
    _vec(stats[1], "rstd", M, torch.float32, dev)
    return stats


def _new_stats(x, stream):
    M = x.shape[0]
    return _empty(M, torch.float32, x.device, stream), _empty(M, torch.float32, x.device, stream)


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
               eps: float = 1e-5, out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """(x - mean) / sqrt(variance + eps) * weight + bias over each row (coalesce_layer_norm).

    ``x`` is a residual stream: float32, or of the result's type.  ``weight``
    and ``bias`` are float32 or of the result's type, both of the same.
    """
    return _norm(x, None, weight, bias, eps, 0.0, 0, 0, out_dtype, out, None, False, None, stream)[0]


def layer_norm_train(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                     eps: float = 1e-5, out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
                     stats: Optional[Tuple[torch.Tensor, torch.Tensor]] = None,
                     stream=None) -> Tuple[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]]:
    """(y, (mean, rstd)): layer_norm and the statistics that
    layer_norm_backward needs, float32, one per row (NaN without columns)."""
    y, _, stats = _norm(x, None, weight, bias, eps, 0.0, 0, 0, out_dtype, out, None, False,
                        True if stats is None else stats, stream)
    return y, stats


def add_layer_norm(x: torch.Tensor, residual: torch.Tensor, weight: Optional[torch.Tensor] = None,
                   bias: Optional[torch.Tensor] = None, eps: float = 1e-5, p: float = 0.0, seed: Seed = 0,
                   offset: int = 0, out: Optional[torch.Tensor] = None, sum_out: Optional[torch.Tensor] = None,
                   stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(y, s): s = residual + dropout(x) and y = layer_norm(s), in one kernel.

    The stream ``residual`` is float32 or of x's type, and so is s, which may be
    formed in place (``sum_out=residual``); y is of x's type, computed from the
    sum before its rounding.  The mask is that of :func:`dropout` with the same
    ``p``, ``seed`` and ``offset``.
    """
    return _norm(x, residual, weight, bias, eps, p, seed, offset, None, out, sum_out, True, None, stream)[:2]


def add_layer_norm_train(x: torch.Tensor, residual: torch.Tensor, weight: Optional[torch.Tensor] = None,
                         bias: Optional[torch.Tensor] = None, eps: float = 1e-5, p: float = 0.0, seed: Seed = 0,
                         offset: int = 0, out: Optional[torch.Tensor] = None, sum_out: Optional[torch.Tensor] = None,
                         stats: Optional[Tuple[torch.Tensor, torch.Tensor]] = None, stream=None):
    """(y, s, (mean, rstd)): add_layer_norm and the statistics that
    layer_norm_backward (of s) needs."""
    return _norm(x, residual, weight, bias, eps, p, seed, offset, None, out, sum_out, True,
                 True if stats is None else stats, stream)


def _like(x, dtype, stream):
    """A result of x's shape, or None where x is no matrix on a GPU (the checks of the call say so)."""
    if x.is_cuda and x.dim() == 2 and dtype in _DTYPES:
        return _new(*x.shape, dtype, x.device, stream)
    return None


def _sum_like(x, residual, stream):
    M, N, _, dev = _rows(x, "x")
    _mat(residual, "residual", M, N, residual.dtype if residual.dtype is torch.float32 else x.dtype, dev)
    return _new(M, N, residual.dtype, residual.device, stream)


def _norm(x, residual, weight, bias, eps, p, seed, offset, out_dtype, out, sum_out, add, stats, stream):
    """(y, sum, (mean, rstd)); stats: None for none, True for new ones."""
    if stream is not None and out is None:
        out = _like(x, x.dtype if add or out_dtype is None else out_dtype, stream)
    if stream is not None and add and sum_out is None:
        sum_out = _sum_like(x, residual, stream)
    if stream is not None and stats is True:
        _rows(x, "x")
        stats = _new_stats(x, stream)
    made = stats is None or stats is True
    if x.is_cuda and (not add or residual is not None) and (made or len(stats) == 2):
        mean, rstd = (stats, stats) if made else stats
        got = _short("layer_norm", "coalesce_layer_norm", stream, x, residual, True if add and sum_out is None else sum_out,
                     weight, bias, True if out is None else out, mean, rstd,
                     -1 if out_dtype is None else _DTYPES.get(out_dtype, -2), eps, p, seed, offset)
        if got is not None:
            _check(got[0])
            return got[1], got[2], got[3:]
    M, N, ldx, dev = _rows(x, "x")
    if _current_device() != dev:
        return _there(dev, _norm, x, residual, weight, bias, eps, p, seed, offset, out_dtype, out, sum_out, add, stats,
                      stream)
    if add:
        dt, sdt = x.dtype, residual.dtype
    else:
        sdt = x.dtype
        dt = out_dtype if out_dtype is not None else out.dtype if out is not None else sdt
    if dt not in _DTYPES or (sdt is not torch.float32 and sdt is not dt):
        raise ValueError("the stream must be float32 or of the result's type, not %s for %s" % (sdt, dt))
    wt = _affine(weight, bias, N, dt, dev)
    mask = _mask(p, seed, offset, dev)
    ldr = lds = 0
    if add:
        if sum_out is None:
            sum_out = _sum_like(x, residual, stream)
        ldr = _mat(residual, "residual", M, N, sdt, dev)
        lds = _mat(sum_out, "sum_out", M, N, sdt, dev)
    if stats is True:
        stats = _new_stats(x, stream)
    mean, rstd = (None, None) if stats is None else _stats(stats, M, dev)
    if out is None:
        out = _new(M, N, dt, x.device, stream)
    ldy = _mat(out, "out", M, N, dt, dev)
    _check(load_library().coalesce_layer_norm(
        x.data_ptr(), ldx, _ptr(residual), ldr, _ptr(sum_out), lds, _ptr(weight), _ptr(bias), out.data_ptr(), ldy,
        _ptr(mean), _ptr(rstd), M, N, _DTYPES[dt], _DTYPES[sdt], _DTYPES[wt], float(eps), *mask,
        _raw_stream(stream, dev)))
    if N == 0:  # the call did nothing
        with torch.cuda.stream(None if stream is None else _stream_object(stream, x.device)):
            for t in (mean, rstd):
                if t is not None:
                    t.fill_(float("nan"))
    return out, sum_out, (mean, rstd)


@functools.lru_cache(maxsize=None)
def _short_size() -> int:
    """The address of coalesce_layer_norm_backward_workspace_size."""
    return ctypes.cast(load_library().coalesce_layer_norm_backward_workspace_size, ctypes.c_void_p).value


def layer_norm_backward(x: torch.Tensor, weight: Optional[torch.Tensor], stats: Tuple[torch.Tensor, torch.Tensor],
                        dout: torch.Tensor, dsum: Optional[torch.Tensor] = None, p: float = 0.0, seed: Seed = 0,
                        offset: int = 0, want_dx: bool = True, want_dbranch: bool = False, want_dweight: bool = True,
                        want_dbias: bool = True, grad_dtype: torch.dtype = torch.float32,
                        dx: Optional[torch.Tensor] = None, dbranch: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None) -> NormGrads:
    """Gradients of layer_norm(x), or of add_layer_norm with the sum ``x``, for
    the upstream gradient ``dout`` (coalesce_layer_norm_backward).

    ``stats`` is what the training forward gave.  ``dsum`` is the gradient that
    arrives along the stream, of x's type (may be ``dx``, which is then formed in
    place).  dx is that of x; dbranch, of dout's type, is dx through the dropout
    of ``p``, ``seed`` and ``offset`` (rounded by itself, not from dx).
    dweight and dbias are of ``grad_dtype``: float32 or dout's.
    """
    if stream is None and x.is_cuda and len(stats) == 2:
        got = _short("layer_norm_backward", "coalesce_layer_norm_backward", None, _short_size(), x, weight, stats[0],
                     stats[1], dout, dsum, dx, dbranch, workspace, want_dx, want_dbranch, want_dweight, want_dbias,
                     _DTYPES.get(grad_dtype, -1), p, seed, offset)
        if got is not None:
            _check(got[0])
            return NormGrads(*got[1:])
    M, N, ldx, dev = _rows(x, "x")
    if _current_device() != dev:
        return _there(dev, layer_norm_backward, x, weight, stats, dout, dsum, p, seed, offset, want_dx, want_dbranch,
                      want_dweight, want_dbias, grad_dtype, dx, dbranch, workspace, stream)
    sdt, dt = x.dtype, dout.dtype
    if dt not in _DTYPES or (sdt is not torch.float32 and sdt is not dt):
        raise ValueError("the stream must be float32 or of dout's type, not %s for %s" % (sdt, dt))
    if grad_dtype is not torch.float32 and grad_dtype is not dt:
        raise ValueError("grad_dtype must be float32 or dout's dtype")
    ldy = _mat(dout, "dout", M, N, dt, dev)
    wt = _affine(weight, None, N, dt, dev)
    mean, rstd = _stats(stats, M, dev)
    mask = _mask(p, seed, offset, dev)
    ldg = 0 if dsum is None else _mat(dsum, "dsum", M, N, sdt, dev)
    lddx = lddb = 0
    dweight = dbias = None
    if want_dx:
        if dx is None:
            dx = _new(M, N, sdt, x.device, stream)
        lddx = _mat(dx, "dx", M, N, sdt, dev)
    if want_dbranch:
        if dbranch is None:
            dbranch = _new(M, N, dt, x.device, stream)
        lddb = _mat(dbranch, "dbranch", M, N, dt, dev)
    if want_dweight:
        dweight = _empty(N, grad_dtype, x.device, stream)
    if want_dbias:
        dbias = _empty(N, grad_dtype, x.device, stream)
    g = NormGrads(dx if want_dx else None, dbranch if want_dbranch else None, dweight, dbias)
    need = 0
    if want_dweight or want_dbias:
        key = ("norm", M, N, 0, dev)
        need = _ws_sizes.get(key)
        if need is None:
            if len(_ws_sizes) >= 4096:
                _ws_sizes.clear()
            need = _ws_sizes[key] = int(load_library().coalesce_layer_norm_backward_workspace_size(M, N))
    ws, nws, _keep = _take(workspace, need, dev, stream)
    _check(load_library().coalesce_layer_norm_backward(
        x.data_ptr(), ldx, _ptr(weight), mean.data_ptr(), rstd.data_ptr(), dout.data_ptr(), ldy, _ptr(dsum), ldg,
        _ptr(g.dx), lddx, _ptr(g.dbranch), lddb, _ptr(dweight), _ptr(dbias), M, N, _DTYPES[dt], _DTYPES[sdt],
        _DTYPES[wt], _DTYPES[grad_dtype], *mask, ws, nws, _raw_stream(stream, dev)))
    return g


def dropout(x: torch.Tensor, p: float, seed: Seed, offset: int = 0, residual: Optional[torch.Tensor] = None,
            out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """residual + x * keep / (1 - p), the mask from a counter-based generator and
    never stored (coalesce_dropout).

    Element (m, n) is kept where word n % 4 of Philox4x32-10 at counter (n // 4,
    m, offset) under the key ``seed`` is at least round(p 2^32); a dropped element
    is 0 whatever it was.  ``seed`` and ``offset`` are 64-bit integers, or
    ``seed`` is an int64 tensor (seed, offset) on the GPU, read when the kernel
    runs: what a captured graph takes, so that its replays can have masks of
    their own.  The result has the residual's type, x's or float32; ``out``
    may be the residual, or x where they share a type.
    """
    if out is None:
        out = _like(x, x.dtype if residual is None else residual.dtype, stream)
    if out is not None and x.is_cuda:
        status = _short("dropout", "coalesce_dropout", stream, x, residual, out, p, seed, offset)
        if status == 0:
            return out
        if status is not None:
            _check(status)
    M, N, ldx, dev = _rows(x, "x")
    if _current_device() != dev:
        return _there(dev, dropout, x, p, seed, offset, residual, out, stream)
    odt = out.dtype if out is not None else residual.dtype if residual is not None else x.dtype
    if odt is not torch.float32 and odt is not x.dtype:
        raise ValueError("the result must be float32 or of x's type")
    mask = _mask(p, seed, offset, dev)
    ldr = 0 if residual is None else _mat(residual, "residual", M, N, odt, dev)
    if out is None:
        out = _new(M, N, odt, x.device, stream)
    ldy = _mat(out, "out", M, N, odt, dev)
    _check(load_library().coalesce_dropout(x.data_ptr(), ldx, _ptr(residual), ldr, out.data_ptr(), ldy, M, N,
                                           _DTYPES[x.dtype], _DTYPES[odt], *mask, _raw_stream(stream, dev)))
    return out


def dropout_backward(dout: torch.Tensor, p: float, seed: Seed, offset: int = 0, out: Optional[torch.Tensor] = None,
                     stream=None) -> torch.Tensor:
    """The gradient of :func:`dropout` in its x: dout * keep / (1 - p) under the
    same mask (the residual's gradient is dout itself)."""
    return dropout(dout, p, seed, offset, None, out, stream)
