"""The feed-forward operators: gated product, GEMM with residual, gradient clipping.

As the rest of the binding: argument checks and marshalling only, all
arithmetic in ``libcoalesce.so``.  Tensors must live on one device; the calls
run there, on ``stream`` or that device's current stream.  What a call makes
(results, workspace) is allocated for that stream; that ``stream`` has waited
for the inputs is the caller's part.
"""
from __future__ import annotations

import ctypes
import math
import weakref
from typing import Iterable, NamedTuple, Optional, Tuple

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import (ACT_NONE, NORM_2, NORM_INF, _ACTS, _DTYPES, _check, _empty, _matrix, _ptr, _raw_current_stream,
               _stream, _stream_object, aligned_copy, load_library)


class GemmGrads(NamedTuple):
    """Gradients of :func:`gemm_residual` (``None``: not wanted; the residual's is ``dout`` itself)."""
    dA: Optional[torch.Tensor]
    dB: Optional[torch.Tensor]
    dbias: Optional[torch.Tensor]


class GatedGrads(NamedTuple):
    """Gradients of :func:`gated_gemm` (``None``: not wanted)."""
    dA: Optional[torch.Tensor]
    dBg: Optional[torch.Tensor]
    dBu: Optional[torch.Tensor]
    dbias_g: Optional[torch.Tensor]
    dbias_u: Optional[torch.Tensor]


def _current_device() -> int:
    return torch._C._cuda_getDevice() if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device()


def _raw_stream(stream, dev: int):
    """The raw handle of `stream`, or of device dev's current stream."""
    if stream is None and _raw_current_stream is not None:
        return _raw_current_stream(dev)
    return _stream(stream)


def _act(act):
    if act not in _ACTS:
        raise ValueError("unknown activation %r" % (act,))
    return _ACTS[act]


def _first(A: torch.Tensor):
    """(rows, cols, pitch, device) of the operand that the others go by."""
    rows, cols, ld = _matrix(A, "A")
    if A.dtype not in _DTYPES:
        raise ValueError("A must be float16 or bfloat16")
    return rows, cols, ld if rows > 1 else _row_pitch(cols, A.dtype), A.get_device()


def _row_pitch(cols: int, dtype: torch.dtype) -> int:
    """A single row has no pitch: it gets the next multiple of 16 bytes."""
    return max(4, (cols + 3) & -4) if dtype is torch.float32 else max(8, (cols + 7) & -8)


def _mat(t: torch.Tensor, name: str, rows: int, cols: int, dtype: torch.dtype, dev: int) -> int:
    """The pitch of a rows x cols operand of `dtype` on device dev (checks only
    what a call needs, in the order that costs least)."""
    if t.shape != (rows, cols) or t.dtype is not dtype or t.get_device() != dev:
        raise ValueError("%s must be a %d x %d tensor of %s on GPU %d, not %s of %s on %s" % (
            name, rows, cols, dtype, dev, tuple(t.shape), t.dtype, t.device))
    st = t.stride()
    if cols > 1 and st[1] != 1:
        raise ValueError("%s must have unit inner stride (row-major)" % name)
    return st[0] if rows > 1 else _row_pitch(cols, dtype)


def _vec(t: Optional[torch.Tensor], name: str, n: int, dtype: torch.dtype, dev: int):
    if t is not None and (t.shape != (n,) or t.dtype is not dtype or not t.is_contiguous() or t.get_device() != dev):
        raise ValueError("%s must be a contiguous length-%d vector of %s on GPU %d" % (name, n, dtype, dev))


def _one_pitch(ts, names, rows: int, cols: int, dtype: torch.dtype, dev: int) -> int:
    """The pitch that two tensors of one shape and type share."""
    if len(ts) != 2:
        raise ValueError("%s must be two tensors" % " and ".join(names))
    ld = _mat(ts[0], names[0], rows, cols, dtype, dev)
    if _mat(ts[1], names[1], rows, cols, dtype, dev) != ld:
        raise ValueError("%s must have one row pitch" % " and ".join(names))
    return ld


def _cols(B: torch.Tensor, name: str) -> int:
    if B.dim() != 2:
        raise ValueError("%s must be 2-D" % name)
    return B.shape[1]


# Workspace sizes by (function, extents, device): a user's shapes repeat.
_ws_sizes = {}


def _workspace(name: str, dev: int, M: int, N: int, K: int, workspace, stream):
    key = (name, M, N, K, dev)
    need = _ws_sizes.get(key)
    if need is None:
        if len(_ws_sizes) >= 4096:
            _ws_sizes.clear()
        need = _ws_sizes[key] = int(getattr(load_library(), name)(M, N, K))
    return _take(workspace, need, dev, stream)


def _take(workspace, need: int, dev: int, stream):
    """(pointer, bytes, tensor to keep alive) of the workspace given, or of one made here."""
    if workspace is None:
        if need == 0:
            return None, 0, None
        workspace = _empty(need, torch.uint8, "cuda", stream, result=False)  # the current device is dev here
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on GPU %d" % dev)
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _new(rows: int, cols: int, dtype, device, stream):
    ld = _row_pitch(cols, dtype)
    t = _empty((rows, ld), dtype, device, stream)
    return t if ld == cols else t[:, :cols]


# The short ways of the compiled extension: (function, address of the entry point).
_short_ways = {}


def _short(name: str, entry: str, stream, *operands):
    """The status of an entry point called by the compiled extension, which reads
    the operands itself; None where one is not as it should be, or the extension is
    not built: the checks in Python then say what is wrong, or make the call."""
    way = _short_ways.get(entry)
    if way is None:
        try:
            from . import _marshal
            way = getattr(_marshal, name), ctypes.cast(getattr(load_library(), entry), ctypes.c_void_p).value
        except (ImportError, AttributeError):
            return None
        _short_ways[entry] = way
    dev = _current_device()
    return way[0](way[1], dev, _raw_stream(stream, dev) or 0, *operands)


def _there(dev: int, call, *args):
    """call(*args) with device dev, not the current one, made current."""
    with torch.cuda.device(dev):
        return call(*args)


def gemm_residual(A: torch.Tensor, B: torch.Tensor, residual: Optional[torch.Tensor] = None,
                  bias: Optional[torch.Tensor] = None, act="none", out_dtype: Optional[torch.dtype] = None,
                  out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """Y = act(A @ B + bias) + residual in one fused kernel (coalesce_gemm_residual).

    The residual has the output's dtype (A's or float32) and may be ``out``
    itself, which is then updated in place.
    """
    return _gemm_residual(A, B, residual, bias, act, out_dtype, out, None, workspace, stream)


def gemm_residual_train(A: torch.Tensor, B: torch.Tensor, residual: Optional[torch.Tensor] = None,
                        bias: Optional[torch.Tensor] = None, act="none", out_dtype: Optional[torch.dtype] = None,
                        out: Optional[torch.Tensor] = None, preact: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None):
    """(Y, Z): gemm_residual and the pre-activation Z = A @ B + bias that
    gemm_residual_backward needs, in A's dtype."""
    if preact is None:
        preact = _new(_first(A)[0], _cols(B, "B"), A.dtype, A.device, stream)
    Y = _gemm_residual(A, B, residual, bias, act, out_dtype, out, preact, workspace, stream)
    return Y, preact


def _out_dtype(A, residual, out_dtype, out):
    if out_dtype is not None:
        return out_dtype
    return out.dtype if out is not None else residual.dtype if residual is not None else A.dtype


def _gemm_residual(A, B, residual, bias, act, out_dtype, out, preact, workspace, stream):
    M, K, lda, dev = _first(A)
    if _current_device() != dev:
        return _there(dev, _gemm_residual, A, B, residual, bias, act, out_dtype, out, preact, workspace, stream)
    N, dt = _cols(B, "B"), A.dtype
    ldb = _mat(B, "B", K, N, dt, dev)
    if bias is not None:
        _vec(bias, "bias", N, dt, dev)
    odt = _out_dtype(A, residual, out_dtype, out)
    if out is None:
        out = _new(M, N, odt, A.device, stream)
    ldy = _mat(out, "out", M, N, odt, dev)
    ldr = 0 if residual is None else _mat(residual, "residual", M, N, odt, dev)
    ldz = 0 if preact is None else _mat(preact, "preact", M, N, dt, dev)
    ws, nws, _keep = _workspace("coalesce_gemm_residual_workspace_size", dev, M, N, K, workspace, stream)
    _check(load_library().coalesce_gemm_residual(
        A.data_ptr(), lda, B.data_ptr(), ldb, _ptr(bias), _ptr(residual), ldr, _ptr(preact), ldz, out.data_ptr(), ldy,
        M, N, K, _DTYPES[dt], _DTYPES[odt], _act(act), ws, nws, _raw_stream(stream, dev)))
    return out


def gated_gemm(A: torch.Tensor, Bg: torch.Tensor, Bu: torch.Tensor, bias_g: Optional[torch.Tensor] = None,
               bias_u: Optional[torch.Tensor] = None, act="silu", out_dtype: Optional[torch.dtype] = None,
               out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """act(A @ Bg + bias_g) * (A @ Bu + bias_u) in one fused kernel (coalesce_gated_gemm).

    Bg and Bu may be the two halves ``W[:, :N]`` and ``W[:, N:]`` of one matrix.
    """
    return _gated_gemm(A, Bg, Bu, bias_g, bias_u, act, out_dtype, out, None, workspace, stream)


def gated_gemm_train(A: torch.Tensor, Bg: torch.Tensor, Bu: torch.Tensor, bias_g: Optional[torch.Tensor] = None,
                     bias_u: Optional[torch.Tensor] = None, act="silu", out_dtype: Optional[torch.dtype] = None,
                     out: Optional[torch.Tensor] = None,
                     preact: Optional[Tuple[torch.Tensor, torch.Tensor]] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None):
    """(H, (Zg, Zu)): gated_gemm and the two pre-activations that
    gated_gemm_backward needs, in A's dtype and of one row pitch."""
    if preact is None:
        M, N = _first(A)[0], _cols(Bg, "Bg")
        preact = tuple(_new(M, N, A.dtype, A.device, stream) for _ in range(2))
    H = _gated_gemm(A, Bg, Bu, bias_g, bias_u, act, out_dtype, out, preact, workspace, stream)
    return H, tuple(preact)


_PREACT = ("preact[0]", "preact[1]")


def _gated_gemm(A, Bg, Bu, bias_g, bias_u, act, out_dtype, out, preact, workspace, stream):
    M, K, lda, dev = _first(A)
    if _current_device() != dev:
        return _there(dev, _gated_gemm, A, Bg, Bu, bias_g, bias_u, act, out_dtype, out, preact, workspace, stream)
    N, dt = _cols(Bg, "Bg"), A.dtype
    ldb = _one_pitch((Bg, Bu), ("Bg", "Bu"), K, N, dt, dev)
    if bias_g is not None:
        _vec(bias_g, "bias_g", N, dt, dev)
    if bias_u is not None:
        _vec(bias_u, "bias_u", N, dt, dev)
    odt = _out_dtype(A, None, out_dtype, out)
    if out is None:
        out = _new(M, N, odt, A.device, stream)
    ldy = _mat(out, "out", M, N, odt, dev)
    zg = zu = None
    ldz = 0
    if preact is not None:
        ldz = _one_pitch(preact, _PREACT, M, N, dt, dev)
        zg, zu = preact[0].data_ptr(), preact[1].data_ptr()
    ws, nws, _keep = _workspace("coalesce_gated_gemm_workspace_size", dev, M, N, K, workspace, stream)
    _check(load_library().coalesce_gated_gemm(
        A.data_ptr(), lda, Bg.data_ptr(), Bu.data_ptr(), ldb, _ptr(bias_g), _ptr(bias_u), zg, zu, ldz, out.data_ptr(),
        ldy, M, N, K, _DTYPES[dt], _DTYPES[odt], _act(act), ws, nws, _raw_stream(stream, dev)))
    return out


def _dout(dout: torch.Tensor, A: torch.Tensor, M: int, N: int, dev: int) -> int:
    return _mat(dout, "dout", M, N, dout.dtype if dout.dtype is torch.float32 else A.dtype, dev)


def _grad_dtype(grad_dtype, A):
    if grad_dtype is not torch.float32 and grad_dtype is not A.dtype:
        raise ValueError("grad_dtype must be float32 or A's dtype")
    return _DTYPES[grad_dtype]


def gemm_residual_backward(A: torch.Tensor, B: torch.Tensor, dout: torch.Tensor,
                           preact: Optional[torch.Tensor] = None, act="none", want_dA: bool = True,
                           want_dB: bool = True, want_dbias: bool = False,
                           grad_dtype: torch.dtype = torch.float32, dA: Optional[torch.Tensor] = None,
                           dB: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                           stream=None) -> GemmGrads:
    """Gradients of gemm_residual for the upstream gradient ``dout`` (A's dtype
    or float32): dA in A's dtype, dB and dbias in ``grad_dtype`` (float32 or
    A's dtype).  ``preact`` is what gemm_residual_train stored; without an
    activation it is not needed."""
    M, K, lda, dev = _first(A)
    if _current_device() != dev:
        return _there(dev, gemm_residual_backward, A, B, dout, preact, act, want_dA, want_dB, want_dbias, grad_dtype,
                      dA, dB, workspace, stream)
    N, dt = _cols(B, "B"), A.dtype
    ldb = _mat(B, "B", K, N, dt, dev)
    ldd = _dout(dout, A, M, N, dev)
    a, gd = _act(act), _grad_dtype(grad_dtype, A)
    if a != ACT_NONE and preact is None:
        raise ValueError("the backward of an activation needs the stored pre-activation")
    ldz = 0 if preact is None else _mat(preact, "preact", M, N, dt, dev)
    ldda = lddb = 0
    dbias = None
    if want_dA:
        if dA is None:
            dA = _new(M, K, dt, A.device, stream)
        ldda = _mat(dA, "dA", M, K, dt, dev)
    if want_dB:
        if dB is None:
            dB = _new(K, N, grad_dtype, A.device, stream)
        lddb = _mat(dB, "dB", K, N, grad_dtype, dev)
    if want_dbias:
        dbias = _empty(N, grad_dtype, A.device, stream)
    g = GemmGrads(dA if want_dA else None, dB if want_dB else None, dbias)
    ws, nws, _keep = _workspace("coalesce_gemm_residual_backward_workspace_size", dev, M, N, K, workspace, stream)
    _check(load_library().coalesce_gemm_residual_backward(
        A.data_ptr(), lda, B.data_ptr(), ldb, _ptr(preact), ldz, dout.data_ptr(), ldd, _ptr(g.dA), ldda, _ptr(g.dB),
        lddb, _ptr(dbias), M, N, K, _DTYPES[dt], _DTYPES[dout.dtype], gd, a, ws, nws, _raw_stream(stream, dev)))
    return g


def gated_gemm_backward(A: torch.Tensor, Bg: torch.Tensor, Bu: torch.Tensor,
                        preact: Tuple[torch.Tensor, torch.Tensor], dout: torch.Tensor, act="silu",
                        want_dA: bool = True, want_dB: bool = True, want_dbias: bool = False,
                        grad_dtype: torch.dtype = torch.float32, dA: Optional[torch.Tensor] = None,
                        dB: Optional[Tuple[torch.Tensor, torch.Tensor]] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None) -> GatedGrads:
    """Gradients of gated_gemm for the upstream gradient ``dout`` (A's dtype or
    float32), from the pre-activations that gated_gemm_train stored: dA in A's
    dtype, dBg, dBu and the bias gradients in ``grad_dtype``."""
    M, K, lda, dev = _first(A)
    if _current_device() != dev:
        return _there(dev, gated_gemm_backward, A, Bg, Bu, preact, dout, act, want_dA, want_dB, want_dbias, grad_dtype,
                      dA, dB, workspace, stream)
    N, dt = _cols(Bg, "Bg"), A.dtype
    ldb = _one_pitch((Bg, Bu), ("Bg", "Bu"), K, N, dt, dev)
    ldd = _dout(dout, A, M, N, dev)
    ldz = _one_pitch(preact, _PREACT, M, N, dt, dev)
    a, gd = _act(act), _grad_dtype(grad_dtype, A)
    ldda = lddb = 0
    dW, db = (None, None), (None, None)
    if want_dA:
        if dA is None:
            dA = _new(M, K, dt, A.device, stream)
        ldda = _mat(dA, "dA", M, K, dt, dev)
    if want_dB:
        dW = dB if dB is not None else tuple(_new(K, N, grad_dtype, A.device, stream) for _ in range(2))
        lddb = _one_pitch(dW, ("dB[0]", "dB[1]"), K, N, grad_dtype, dev)
    if want_dbias:
        db = _empty(N, grad_dtype, A.device, stream), _empty(N, grad_dtype, A.device, stream)
    g = GatedGrads(dA if want_dA else None, dW[0], dW[1], db[0], db[1])
    ws, nws, _keep = _workspace("coalesce_gated_gemm_backward_workspace_size", dev, M, N, K, workspace, stream)
    _check(load_library().coalesce_gated_gemm_backward(
        A.data_ptr(), lda, Bg.data_ptr(), Bu.data_ptr(), ldb, preact[0].data_ptr(), preact[1].data_ptr(), ldz,
        dout.data_ptr(), ldd, _ptr(g.dA), ldda, _ptr(dW[0]), _ptr(dW[1]), lddb, _ptr(db[0]), _ptr(db[1]), M, N, K,
        _DTYPES[dt], _DTYPES[dout.dtype], gd, a, ws, nws, _raw_stream(stream, dev)))
    return g


# ---------------------------------------------------------------------------
# Gradient norm and clipping
# ---------------------------------------------------------------------------

def _held(tensors, stream):
    """`tensors` as a list or tuple.  Those of a generator may be made as it
    runs and live only in the list: it has to outlive the launch, and `stream`
    has to wait for them, as no caller could tell it to."""
    if tensors is None or isinstance(tensors, (list, tuple)):
        return tensors
    tensors = list(tensors)
    if stream is not None:
        for t in tensors:
            if isinstance(t, torch.Tensor) and t.is_cuda:
                on, here = _stream_object(stream, t.device), torch.cuda.current_stream(t.device)
                if on != here:
                    on.wait_stream(here)
                    t.record_stream(on)
    return tensors


def _grad_list(tensors, out):
    """(count, device, sources, destinations, sizes, types, columns, pitches,
    pitches of the destinations): the host arrays of the C call (bytes objects,
    to be kept alive until it returns; the last three None for a list of dense
    tensors)."""
    try:
        from ._marshal import grad_list
    except ImportError as e:
        raise RuntimeError("%s is not built (python -m mlp_megakernel_amd.build)" % e.name) from None
    n, dev, *arrays = grad_list(tensors, out)
    return (n, _current_device() if n == 0 else dev, *arrays)


def _norm_code(norm_type) -> int:
    if norm_type == 2:
        return NORM_2
    if norm_type == math.inf or norm_type == "inf":
        return NORM_INF
    raise ValueError("norm_type must be 2 or inf")


def _norm_out(norm, dev, stream):
    if norm is None:
        norm = _empty((), torch.float32, "cuda", stream)  # the current device is dev here
    elif norm.numel() != 1 or norm.dtype is not torch.float32 or norm.get_device() != dev:
        raise ValueError("norm must be one float32 on GPU %d" % dev)
    return norm


def grad_norm(tensors: Iterable[torch.Tensor], norm_type=2.0, norm: Optional[torch.Tensor] = None,
              workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The 2-norm or largest magnitude (``norm_type`` inf) of all the tensors
    taken as one vector, as a float32 scalar on their device (coalesce_grad_norm)."""
    tensors = _held(tensors, stream)
    return _norm_call(_grad_list(tensors, None), None, norm_type, norm, workspace, stream)


def clip_grad_norm(tensors: Iterable[torch.Tensor], max_norm: float, norm_type=2.0,
                   out: Optional[Iterable[torch.Tensor]] = None, norm: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Scale gradients so that their global norm is at most ``max_norm``
    (coalesce_clip_grad_norm) and return the norm they had, a float32 scalar on
    their device.  In place, or into ``out`` (one tensor per gradient, of its
    size, memory order and dtype).  Nothing synchronises with the host; tensors of
    several dtypes may be mixed.  A tensor is dense or a matrix of unit inner
    stride, as the gradients of :func:`gated_gemm_backward` are."""
    tensors, out = _held(tensors, stream), _held(out, stream)
    return _norm_call(_grad_list(tensors, out), float(max_norm), norm_type, norm, workspace, stream)


def _norm_call(lists, max_norm, norm_type, norm, workspace, stream):
    n, dev, src, dst, numel, dts, cols, ld, ld_out = lists
    if _current_device() != dev:
        return _there(dev, _norm_call, lists, max_norm, norm_type, norm, workspace, stream)
    lib, code = load_library(), _norm_code(norm_type)
    norm = _norm_out(norm, dev, stream)
    need = int(lib.coalesce_grad_norm_rows_workspace_size(numel, cols, dts, n))
    ws, nws, _keep = _take(workspace, need, dev, stream)
    if max_norm is None:
        _check(lib.coalesce_grad_norm_rows(src, numel, cols, ld, dts, n, code, norm.data_ptr(), ws, nws,
                                           _raw_stream(stream, dev)))
    else:
        _check(lib.coalesce_clip_grad_norm_rows(src, dst, numel, cols, ld, ld_out, dts, n, code, max_norm,
                                                norm.data_ptr(), ws, nws, _raw_stream(stream, dev)))
    return norm


# ---------------------------------------------------------------------------
# Modules
# ---------------------------------------------------------------------------

from .int8 import gated_gemm_int8, gemm_int8, quantize_columns, quantize_rows  # noqa: E402 (they use what is above)
from .norm import dropout as _dropout  # noqa: E402
from .norm import dropout_backward, layer_norm, layer_norm_backward, layer_norm_train  # noqa: E402


def _rows16(t: torch.Tensor) -> torch.Tensor:
    """`t` with 16-byte aligned rows and unit inner stride (a copy if it has not)."""
    es = t.element_size()
    if t.dim() == 2 and (t.stride(1) == 1 or t.shape[1] == 1) and t.data_ptr() % 16 == 0 and \
            (t.stride(0) * es) % 16 == 0 and t.stride(0) >= t.shape[1]:
        return t
    return aligned_copy(t, t.device)


def _vec16(t: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    """`t` contiguous and 16-byte aligned (a copy if it is not, as a slice of a flat buffer need not be)."""
    if t is None or (t.data_ptr() % 16 == 0 and t.is_contiguous()):
        return t
    return t.clone(memory_format=torch.contiguous_format)


class _EagerGraph:
    """Held by an autograd node made outside a capture, on the default stream:
    the tensors that its graph's leaves are."""
    alive = weakref.WeakSet()

    def __init__(self, tensors):
        self.leaves = [weakref.ref(t) for t in tensors if t is not None and t.requires_grad and t.is_leaf]
        self.alive.add(self)

    @classmethod
    def refuse_capture(cls, tensors):
        """While such a graph lives, autograd adds to its leaves' gradients on the
        default stream.  A captured backward would make that stream, which
        cannot be captured, wait for the capturing one: the process ends."""
        for g in list(cls.alive):
            if any(r() is t for r in g.leaves for t in tensors):
                raise RuntimeError("an autograd graph of the same leaves, made on the default stream, is still alive: "
                                   "drop its outputs before the capture, or warm up on the stream of the capture")


def _refuse_recorded(tensors, what="GatedFFN", trace="GatedFFN without gradients cannot be traced: trace it with "
                                                      "gradients enabled"):
    """The plain calls are no torch operations: what records those would miss
    them, a tangent be lost and a trace return memory that nothing wrote."""
    if torch.jit.is_tracing():
        raise RuntimeError(trace)
    if getattr(forward_ad, "_current_level", 0) >= 0 and \
            any(t is not None and forward_ad.unpack_dual(t).tangent is not None for t in tensors):
        raise NotImplementedError("%s has no forward-mode derivative" % what)


def _draw_seed(device) -> torch.Tensor:
    """(seed, offset) of a dropout mask, from torch's generator of the device: it
    goes by torch.manual_seed, and a captured graph draws anew at every replay."""
    return torch.randint(-2 ** 63, 2 ** 63 - 1, (2,), device=device, dtype=torch.int64)


def _down(H, Wd, bd, skip, p, seed):
    """skip + dropout(H Wd + bd); without a dropout in the product's own epilogue.

    With one H Wd + bd is rounded to the type in between, half a step of its own more
    than in the epilogue: the dropout reads what a product of that type gives, and an
    fp32 one would cost it 4 more bytes an element written and read.
    """
    if seed is None:
        return gemm_residual(H, Wd, skip, bd)
    h = gemm_residual(H, Wd, None, bd)
    return _dropout(h, p, seed, residual=skip, out=h)


class _GatedFFNFunction(torch.autograd.Function):
    """x + dropout((act(n Wg + bg) * (n Wu + bu)) Wd + bd) as one autograd node, n = x or its layer norm."""

    @staticmethod
    def forward(ctx, graph, x, act, residual, norm, eps, p, seed, Wg, Wu, Wd, bg, bu, bd, nw, nb):
        n, stats = (x, (None, None)) if not norm else layer_norm_train(x, nw, nb, eps)
        H, (Zg, Zu) = gated_gemm_train(n, Wg, Wu, bg, bu, act=act)
        y = _down(H, Wd, bd, x if residual else None, p, seed)
        ctx.act, ctx.residual, ctx.norm, ctx.p, ctx.graph = act, residual, norm, p, graph
        ctx.save_for_backward(x, n, Wg, Wu, Wd, Zg, Zu, H, nw, seed, *stats)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, n, Wg, Wu, Wd, Zg, Zu, H, nw, seed, *stats = ctx.saved_tensors
        need_x = ctx.needs_input_grad[1]
        need = dict(zip(("Wg", "Wu", "Wd", "bg", "bu", "bd", "nw", "nb"), ctx.needs_input_grad[8:]))
        dy = _rows16(dy.to(x.dtype))
        dh = dy if seed is None else dropout_backward(dy, ctx.p, seed)
        # dH is rounded to the type as H was: it is an operand of the next products'
        # dZ.  The skip's dy joins dx after dx's own rounding, a second half step (with a
        # norm in its backward, before the one rounding).
        down = gemm_residual_backward(H, Wd, dh, want_dB=need["Wd"], want_dbias=need["bd"], grad_dtype=Wd.dtype)
        up = gated_gemm_backward(n, Wg, Wu, (Zg, Zu), down.dA, act=ctx.act,
                                 want_dA=need_x or need["nw"] or need["nb"], want_dB=need["Wg"] or need["Wu"],
                                 want_dbias=need["bg"] or need["bu"], grad_dtype=Wg.dtype)
        dx, dnw, dnb = up.dA, None, None
        if ctx.norm:
            if dx is not None:
                g = layer_norm_backward(x, nw, stats, dx, dy if ctx.residual else None, want_dx=need_x,
                                        want_dweight=need["nw"], want_dbias=need["nb"], grad_dtype=nw.dtype)
                dx, dnw, dnb = g.dx, g.dweight, g.dbias
        elif need_x and ctx.residual:
            dx = dx + dy
        return (None, dx, None, None, None, None, None, None, up.dBg, up.dBu, down.dB, up.dbias_g, up.dbias_u,
                down.dbias, dnw, dnb)


class GatedFFN(torch.nn.Module):
    """The gated feed-forward block ``y = x + dropout((act(n Wg + bg) * (n Wu + bu)) Wd + bd)``.

    Weights in the x @ W orientation.  ``residual=False`` leaves out the
    ``x +``, ``bias=False`` (the default) the biases.  x is ``[..., D]``.  n is x,
    or with ``norm=True`` its layer norm (over the last dimension, ``eps``, with
    weight and bias).  ``dropout`` is the probability that an element is dropped
    while the module trains; the mask is never stored, its seed comes from torch's
    generator of the device.  :meth:`quantized` gives the block with 8-bit weights.

    The forward and backward can be captured in a graph after a warm-up on a
    side stream; a capture while an autograd graph that a GatedFFN made of the
    same leaves on the default stream is alive raises an error (graphs that other
    operations made of them there are not seen: drop those first).  So do
    second derivatives, forward-mode ones and torch.jit.trace without gradients.

    Widths that are no multiples of 8 work, but the kernels read rows on 16-byte
    boundaries: the weights of such a block are copied at every call.
    """

    def __init__(self, D: int, H: int, act="silu", bias: bool = False, residual: bool = True, device="cuda",
                 dtype=torch.bfloat16, norm: bool = False, dropout: float = 0.0, eps: float = 1e-5):
        super().__init__()
        _act(act)
        if not 0.0 <= dropout <= 1.0:
            raise ValueError("dropout must lie in [0, 1], not %r" % (dropout,))
        self.act, self.residual, self.D, self.H = act, residual, D, H
        self.norm, self.dropout, self.eps = norm, dropout, eps

        def param(*shape, std=0.0):
            p = torch.nn.Parameter(torch.zeros(*shape, device=device, dtype=dtype))
            if std:
                torch.nn.init.normal_(p, std=std)
            return p

        self.Wg, self.Wu = param(D, H, std=D ** -0.5), param(D, H, std=D ** -0.5)
        self.Wd = param(H, D, std=H ** -0.5)
        self.bg, self.bu, self.bd = (param(H), param(H), param(D)) if bias else (None, None, None)
        self.norm_weight = self.norm_bias = None
        if norm:
            self.norm_weight, self.norm_bias = torch.nn.Parameter(torch.ones(D, device=device, dtype=dtype)), param(D)

    def __setstate__(self, state):
        # modules pickled before there was a norm and a dropout have neither
        for name, value in (("norm", False), ("dropout", 0.0), ("eps", 1e-5), ("norm_weight", None),
                            ("norm_bias", None)):
            if name not in state and name not in state.get("_parameters", {}):
                state[name] = value
        super().__setstate__(state)

    def quantized(self) -> "QuantizedGatedFFN":
        """This block with its weights as they are now in 8 bits, for inference."""
        return QuantizedGatedFFN(self)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        shape = x.shape
        if not shape or shape[-1] != self.D:
            raise ValueError("x must be [..., %d], not %s" % (self.D, tuple(shape)))
        x2 = _rows16(x.reshape(-1, self.D))
        Wg, Wu, Wd = _rows16(self.Wg), _rows16(self.Wu), _rows16(self.Wd)
        bg, bu, bd = _vec16(self.bg), _vec16(self.bu), _vec16(self.bd)
        nw, nb = _vec16(self.norm_weight), _vec16(self.norm_bias)
        p = self.dropout if self.training else 0.0
        if torch.is_grad_enabled() and (x.requires_grad or any(p.requires_grad for p in self.parameters())):
            leaves = (x, *self.parameters())
            graph = None
            if torch.cuda.is_current_stream_capturing():
                _EagerGraph.refuse_capture(leaves)
            elif torch.cuda.current_stream(x.device) == torch.cuda.default_stream(x.device):
                graph = _EagerGraph(leaves)
            seed = _draw_seed(x2.device) if p > 0 else None
            y = _GatedFFNFunction.apply(graph, x2, self.act, self.residual, self.norm, self.eps, p, seed, Wg, Wu, Wd,
                                        bg, bu, bd, nw, nb)
        else:
            _refuse_recorded((x2, Wg, Wu, Wd, bg, bu, bd, nw, nb))
            n = layer_norm(x2, nw, nb, self.eps) if self.norm else x2
            h = gated_gemm(n, Wg, Wu, bg, bu, act=self.act)
            y = _down(h, Wd, bd, x2 if self.residual else None, p, _draw_seed(x2.device) if p > 0 else None)
        return y.reshape(shape)


class QuantizedGatedFFN(torch.nn.Module):
    """A :class:`GatedFFN` for inference with its weights in 8 bits, one scale per
    channel, and the tokens quantised in front of each product, one scale per token.

    Made by :meth:`GatedFFN.quantized`.  x is of the block's type; nothing
    depends on the other tokens of a call.  There is no gradient and no dropout.
    ``half()``, ``bfloat16()``, ``float()`` and ``to(dtype)`` change the type of x
    and of the result alone: weights stay 8-bit, scales and biases float32.
    """

    def __init__(self, block: GatedFFN):
        super().__init__()
        self.act, self.residual, self.norm, self.eps = block.act, block.residual, block.norm, block.eps
        self.D, self.H, self.dtype = block.D, block.H, block.Wg.dtype
        with torch.no_grad():
            for name in ("Wg", "Wu", "Wd"):
                q, scale = quantize_columns(_rows16(getattr(block, name).detach()))
                self.register_buffer(name, q)
                self.register_buffer(name + "_scale", scale)
            for name in ("bg", "bu", "bd", "norm_weight", "norm_bias"):
                t = getattr(block, name)
                self.register_buffer(name, None if t is None else t.detach().float().clone())

    def _apply(self, fn, recurse=True):
        dtype = fn(self.Wg_scale.new_empty(1, dtype=self.dtype)).dtype
        if dtype not in _DTYPES:
            raise TypeError("QuantizedGatedFFN takes float32, float16 or bfloat16, not %s" % dtype)

        def moved(t):  # fn without its change of type, which leaves integers as they are
            s = fn(t)
            if s.dtype is t.dtype:
                return s
            s = fn(t.view(torch.uint8))
            if s.dtype is not torch.uint8:
                raise TypeError("the weights of a QuantizedGatedFFN stay 8-bit")
            return s.view(t.dtype)

        super()._apply(moved, recurse)
        self.dtype = dtype
        return self

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        shape = x.shape
        if not shape or shape[-1] != self.D or x.dtype is not self.dtype:
            raise ValueError("x must be [..., %d] of %s, not %s of %s" % (self.D, self.dtype, tuple(shape), x.dtype))
        if torch.is_grad_enabled() and x.requires_grad:
            raise RuntimeError("QuantizedGatedFFN has no gradient")
        x2 = _rows16(x.reshape(-1, self.D))
        _refuse_recorded((x2,), "QuantizedGatedFFN", "QuantizedGatedFFN cannot be traced")
        n = x2
        if self.norm:
            n = layer_norm(x2, _vec16(self.norm_weight), _vec16(self.norm_bias), self.eps)
        q, s = quantize_rows(n)
        h = gated_gemm_int8(q, _rows16(self.Wg), _rows16(self.Wu), s, _vec16(self.Wg_scale), _vec16(self.Wu_scale),
                            _vec16(self.bg), _vec16(self.bu), act=self.act, out_dtype=self.dtype)
        q, s = quantize_rows(h)
        y = gemm_int8(q, _rows16(self.Wd), s, _vec16(self.Wd_scale), _vec16(self.bd), x2 if self.residual else None,
                      out_dtype=self.dtype)
        return y.reshape(shape)
