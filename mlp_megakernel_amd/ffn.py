"""The feed-forward operators: gated product, GEMM with residual, gradient clipping.

As the rest of the binding: argument checks and marshalling only, all
arithmetic in ``libcoalesce.so``.  Tensors must live on one device; the calls
run there, on ``stream`` or that device's current stream.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
from typing import NamedTuple, Optional, Sequence, Tuple

import torch

from . import (ACT_NONE, NORM_2, NORM_INF, _ACTS, _DTYPES, _c_array, _check, _matrix, _ptr, _stream, aligned_copy,
               aligned_empty, load_library)

_i64, _i32, _vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p


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


_NO_GUARD = contextlib.nullcontext()


def _on(device: torch.device):
    """Context in which `device` is the current one."""
    return _NO_GUARD if device.index == torch.cuda.current_device() else torch.cuda.device(device)


def _used_on(stream, *tensors):
    """Tell the allocator that tensors it made here are used on another stream."""
    if stream is None:
        return
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream))
    for t in tensors:
        if t is not None and t.numel():
            t.record_stream(stream)


def _act(act):
    if act not in _ACTS:
        raise ValueError("unknown activation %r" % (act,))
    return _ACTS[act]


def _dtype(t: torch.Tensor, name: str):
    if t.dtype not in _DTYPES:
        raise ValueError("%s must be float32, float16 or bfloat16" % name)
    return _DTYPES[t.dtype]


def _pitched(t: torch.Tensor, name: str):
    """(rows, cols, ld) as _matrix gives them; a single row has no pitch, so
    one of any length gets the next multiple of 16 bytes."""
    rows, cols, ld = _matrix(t, name)
    if rows <= 1:
        per = 16 // t.element_size()
        ld = max(per, (cols + per - 1) // per * per)
    return rows, cols, ld


def _mat(t: torch.Tensor, name: str, like: torch.Tensor, shape=None, dtype=None):
    """The pitch of a 2-D operand on like's device, of the given shape and type."""
    rows, cols, ld = _pitched(t, name)
    if t.device != like.device:
        raise ValueError("%s is on %s, not on %s" % (name, t.device, like.device))
    if shape is not None and (rows, cols) != shape:
        raise ValueError("%s must be %d x %d" % ((name,) + shape))
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s" % (name, dtype))
    return ld


def _vec(t: Optional[torch.Tensor], name: str, like: torch.Tensor, n: int, dtype):
    if t is None:
        return
    if t.dim() != 1 or t.shape[0] != n or t.dtype != dtype or not t.is_contiguous() or t.device != like.device:
        raise ValueError("%s must be a contiguous length-%d vector of %s on %s" % (name, n, dtype, like.device))


def _extents(A: torch.Tensor, Bs, names):
    M, K, lda = _pitched(A, "A")
    if A.dtype not in _DTYPES:
        raise ValueError("A must be float16 or bfloat16")
    N = Bs[0].shape[1] if Bs[0].dim() == 2 else -1
    return M, N, K, lda, _one_pitch(Bs, names, A, (K, N), A.dtype)


def _one_pitch(ts, names, like, shape, dtype):
    """The pitch that tensors of one shape and type share."""
    ld = [_mat(t, n, like, shape, dtype) for t, n in zip(ts, names)]
    if any(x != ld[0] for x in ld):
        raise ValueError("%s must have one row pitch" % " and ".join(names))
    return ld[0]


# Workspace sizes by (function, extents, device): a user's shapes repeat.
_ws_sizes = {}


def _workspace(name: str, device: torch.device, M: int, N: int, K: int, workspace, stream):
    key = (name, M, N, K, device.index)
    need = _ws_sizes.get(key)
    if need is None:
        if len(_ws_sizes) >= 4096:
            _ws_sizes.clear()
        need = _ws_sizes[key] = int(getattr(load_library(), name)(M, N, K))
    return _take(workspace, need, device, stream)


def _take(workspace, need: int, device: torch.device, stream):
    """(pointer, bytes, tensor to keep alive) of the workspace given, or of one made here."""
    if workspace is None:
        if need == 0:
            return None, 0, None
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
        _used_on(stream, workspace)
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on %s" % device)
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _new(rows: int, cols: int, dtype, device, stream):
    t = aligned_empty(rows, cols, dtype, device)
    _used_on(stream, t)
    return t


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
        preact = _new(A.shape[0], B.shape[1], A.dtype, A.device, stream)
    Y = _gemm_residual(A, B, residual, bias, act, out_dtype, out, preact, workspace, stream)
    return Y, preact


def _out_dtype(A, residual, out_dtype, out):
    if out_dtype is not None:
        return out_dtype
    return out.dtype if out is not None else residual.dtype if residual is not None else A.dtype


def _gemm_residual(A, B, residual, bias, act, out_dtype, out, preact, workspace, stream):
    lib = load_library()
    M, N, K, lda, ldb = _extents(A, (B,), ("B",))
    _vec(bias, "bias", A, N, A.dtype)
    odt = _out_dtype(A, residual, out_dtype, out)
    if out is None:
        out = _new(M, N, odt, A.device, stream)
    ldy = _mat(out, "out", A, (M, N), odt)
    ldr = 0 if residual is None else _mat(residual, "residual", A, (M, N), odt)
    ldz = 0 if preact is None else _mat(preact, "preact", A, (M, N), A.dtype)
    with _on(A.device):
        ws, nws, _keep = _workspace("coalesce_gemm_residual_workspace_size", A.device, M, N, K, workspace, stream)
        _check(lib.coalesce_gemm_residual(_ptr(A), lda, _ptr(B), ldb, _ptr(bias), _ptr(residual), ldr, _ptr(preact),
                                          ldz, _ptr(out), ldy, M, N, K, _DTYPES[A.dtype], _dtype(out, "out"),
                                          _act(act), ws, nws, _stream(stream)))
    return out


def gated_gemm(A: torch.Tensor, Bg: torch.Tensor, Bu: torch.Tensor, bias_g: Optional[torch.Tensor] = None,
               bias_u: Optional[torch.Tensor] = None, act="silu", out_dtype: Optional[torch.dtype] = None,
               out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """act(A @ Bg + bias_g) * (A @ Bu + bias_u) in one fused kernel (coalesce_gated_gemm).

    Bg and Bu may be the two halves ``W[:, :N]`` and ``W[:, N:]`` of one matrix.
    """
    return _gated_gemm(A, Bg, Bu, bias_g, bias_u, act, out_dtype, out, (None, None), workspace, stream)


def gated_gemm_train(A: torch.Tensor, Bg: torch.Tensor, Bu: torch.Tensor, bias_g: Optional[torch.Tensor] = None,
                     bias_u: Optional[torch.Tensor] = None, act="silu", out_dtype: Optional[torch.dtype] = None,
                     out: Optional[torch.Tensor] = None,
                     preact: Optional[Tuple[torch.Tensor, torch.Tensor]] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None):
    """(H, (Zg, Zu)): gated_gemm and the two pre-activations that
    gated_gemm_backward needs, in A's dtype and of one row pitch."""
    if preact is None:
        preact = tuple(_new(A.shape[0], Bg.shape[1], A.dtype, A.device, stream) for _ in range(2))
    H = _gated_gemm(A, Bg, Bu, bias_g, bias_u, act, out_dtype, out, preact, workspace, stream)
    return H, tuple(preact)


def _preact_pitch(preact, A, M, N):
    if len(preact) != 2:
        raise ValueError("preact must be the two stored pre-activations")
    return _one_pitch(preact, ("preact[0]", "preact[1]"), A, (M, N), A.dtype)


def _gated_gemm(A, Bg, Bu, bias_g, bias_u, act, out_dtype, out, preact, workspace, stream):
    lib = load_library()
    M, N, K, lda, ldb = _extents(A, (Bg, Bu), ("Bg", "Bu"))
    _vec(bias_g, "bias_g", A, N, A.dtype)
    _vec(bias_u, "bias_u", A, N, A.dtype)
    odt = _out_dtype(A, None, out_dtype, out)
    if out is None:
        out = _new(M, N, odt, A.device, stream)
    ldy = _mat(out, "out", A, (M, N), odt)
    ldz = 0 if preact[0] is None else _preact_pitch(preact, A, M, N)
    with _on(A.device):
        ws, nws, _keep = _workspace("coalesce_gated_gemm_workspace_size", A.device, M, N, K, workspace, stream)
        _check(lib.coalesce_gated_gemm(_ptr(A), lda, _ptr(Bg), _ptr(Bu), ldb, _ptr(bias_g), _ptr(bias_u),
                                       _ptr(preact[0]), _ptr(preact[1]), ldz, _ptr(out), ldy, M, N, K,
                                       _DTYPES[A.dtype], _dtype(out, "out"), _act(act), ws, nws, _stream(stream)))
    return out


def _grad_out(t, name, A, rows, cols, dtype, stream):
    """(tensor, pitch) of a wanted matrix gradient, made here if none is given."""
    if t is None:
        t = _new(rows, cols, dtype, A.device, stream)
    return t, _mat(t, name, A, (rows, cols), dtype)


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
    lib = load_library()
    M, N, K, lda, ldb = _extents(A, (B,), ("B",))
    ldd = _mat(dout, "dout", A, (M, N))
    a = _act(act)
    if a != ACT_NONE and preact is None:
        raise ValueError("the backward of an activation needs the stored pre-activation")
    ldz = 0 if preact is None else _mat(preact, "preact", A, (M, N), A.dtype)
    ldda = lddb = 0
    dbias = None
    if want_dA:
        dA, ldda = _grad_out(dA, "dA", A, M, K, A.dtype, stream)
    if want_dB:
        dB, lddb = _grad_out(dB, "dB", A, K, N, grad_dtype, stream)
    if want_dbias:
        dbias = torch.empty(N, dtype=grad_dtype, device=A.device)
        _used_on(stream, dbias)
    g = GemmGrads(dA if want_dA else None, dB if want_dB else None, dbias)
    with _on(A.device):
        ws, nws, _keep = _workspace("coalesce_gemm_residual_backward_workspace_size", A.device, M, N, K, workspace,
                                    stream)
        _check(lib.coalesce_gemm_residual_backward(_ptr(A), lda, _ptr(B), ldb, _ptr(preact), ldz, _ptr(dout), ldd,
                                                   _ptr(g.dA), ldda, _ptr(g.dB), lddb, _ptr(dbias), M, N, K,
                                                   _DTYPES[A.dtype], _dtype(dout, "dout"), _DTYPES[grad_dtype], a, ws,
                                                   nws, _stream(stream)))
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
    lib = load_library()
    M, N, K, lda, ldb = _extents(A, (Bg, Bu), ("Bg", "Bu"))
    ldd = _mat(dout, "dout", A, (M, N))
    ldz = _preact_pitch(preact, A, M, N)
    ldda = lddb = 0
    dW, db = [None, None], [None, None]
    if want_dA:
        dA, ldda = _grad_out(dA, "dA", A, M, K, A.dtype, stream)
    if want_dB:
        dW = list(dB) if dB is not None else [_new(K, N, grad_dtype, A.device, stream) for _ in range(2)]
        if len(dW) != 2:
            raise ValueError("dB must be two tensors")
        lddb = _one_pitch(dW, ("dB[0]", "dB[1]"), A, (K, N), grad_dtype)
    if want_dbias:
        db = [torch.empty(N, dtype=grad_dtype, device=A.device) for _ in range(2)]
        _used_on(stream, *db)
    g = GatedGrads(dA if want_dA else None, dW[0], dW[1], db[0], db[1])
    with _on(A.device):
        ws, nws, _keep = _workspace("coalesce_gated_gemm_backward_workspace_size", A.device, M, N, K, workspace,
                                    stream)
        _check(lib.coalesce_gated_gemm_backward(_ptr(A), lda, _ptr(Bg), _ptr(Bu), ldb, _ptr(preact[0]),
                                                _ptr(preact[1]), ldz, _ptr(dout), ldd, _ptr(g.dA), ldda, _ptr(dW[0]),
                                                _ptr(dW[1]), lddb, _ptr(db[0]), _ptr(db[1]), M, N, K,
                                                _DTYPES[A.dtype], _dtype(dout, "dout"), _DTYPES[grad_dtype], _act(act),
                                                ws, nws, _stream(stream)))
    return g


# ---------------------------------------------------------------------------
# Gradient norm and clipping
# ---------------------------------------------------------------------------

def _dense(t: torch.Tensor) -> bool:
    """Whether the tensor's elements fill one run of memory, in any order."""
    if t.is_contiguous():
        return True
    n = 1
    for size, st in sorted(((s, st) for s, st in zip(t.shape, t.stride()) if s != 1), key=lambda x: x[1]):
        if st != n:
            return False
        n *= size
    return True


def _grad_list(tensors, out):
    tensors = list(tensors)
    dev = tensors[0].device if tensors else torch.device("cuda", torch.cuda.current_device())
    for i, t in enumerate(tensors):
        if t.device != dev or not t.is_cuda:
            raise ValueError("tensor %d is on %s, not on %s" % (i, t.device, dev))
        if t.dtype not in _DTYPES:
            raise ValueError("tensor %d must be float32, float16 or bfloat16" % i)
        if not _dense(t):
            raise ValueError("tensor %d must be dense (its elements one run of memory)" % i)
    if out is not None:
        if len(out) != len(tensors):
            raise ValueError("out must hold one tensor per gradient")
        for i, (t, o) in enumerate(zip(tensors, out)):
            if o.shape != t.shape or o.dtype != t.dtype or o.device != dev or o.stride() != t.stride():
                raise ValueError("out[%d] must have its gradient's shape, strides, dtype and device" % i)
    src = _c_array(_vp, tuple([t.data_ptr() for t in tensors]))
    numel = _c_array(_i64, tuple([t.numel() for t in tensors]))
    dts = _c_array(_i32, tuple([_DTYPES[t.dtype] for t in tensors]))
    dst = src if out is None else _c_array(_vp, tuple([t.data_ptr() for t in out]))
    return len(tensors), dev, src, dst, numel, dts


def _norm_code(norm_type) -> int:
    if norm_type == 2:
        return NORM_2
    if norm_type == math.inf or norm_type == "inf":
        return NORM_INF
    raise ValueError("norm_type must be 2 or inf")


def _norm_out(norm, dev, stream):
    if norm is None:
        norm = torch.empty((), dtype=torch.float32, device=dev)
        _used_on(stream, norm)
    elif norm.numel() != 1 or norm.dtype != torch.float32 or norm.device != dev:
        raise ValueError("norm must be one float32 on %s" % dev)
    return norm


def grad_norm(tensors: Sequence[torch.Tensor], norm_type=2.0, norm: Optional[torch.Tensor] = None,
              workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The 2-norm or largest magnitude (``norm_type`` inf) of all the tensors
    taken as one vector, as a float32 scalar on their device (coalesce_grad_norm)."""
    lib = load_library()
    n, dev, src, _, numel, dts = _grad_list(tensors, None)
    code = _norm_code(norm_type)
    norm = _norm_out(norm, dev, stream)
    with _on(dev):
        ws, nws, _keep = _take(workspace, int(lib.coalesce_grad_norm_workspace_size(numel, dts, n)), dev, stream)
        _check(lib.coalesce_grad_norm(src, numel, dts, n, code, _ptr(norm), ws, nws, _stream(stream)))
    return norm


def clip_grad_norm(tensors: Sequence[torch.Tensor], max_norm: float, norm_type=2.0,
                   out: Optional[Sequence[torch.Tensor]] = None, norm: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Scale gradients so that their global norm is at most ``max_norm``
    (coalesce_clip_grad_norm) and return the norm they had, a float32 scalar on
    their device.  In place, or into ``out`` (one tensor per gradient, of its
    shape, strides and dtype).  Nothing synchronises with the host; tensors of
    several dtypes may be mixed."""
    lib = load_library()
    n, dev, src, dst, numel, dts = _grad_list(tensors, out)
    code = _norm_code(norm_type)
    norm = _norm_out(norm, dev, stream)
    with _on(dev):
        ws, nws, _keep = _take(workspace, int(lib.coalesce_grad_norm_workspace_size(numel, dts, n)), dev, stream)
        _check(lib.coalesce_clip_grad_norm(src, dst, numel, dts, n, code, float(max_norm), _ptr(norm), ws, nws,
                                           _stream(stream)))
    return norm


# ---------------------------------------------------------------------------
# Module
# ---------------------------------------------------------------------------

def _rows16(t: torch.Tensor) -> torch.Tensor:
    """`t` with 16-byte aligned rows and unit inner stride (a copy if it has not)."""
    es = t.element_size()
    if t.dim() == 2 and (t.stride(1) == 1 or t.shape[1] == 1) and t.data_ptr() % 16 == 0 and \
            (t.stride(0) * es) % 16 == 0 and t.stride(0) >= t.shape[1]:
        return t
    return aligned_copy(t, t.device)


class _GatedFFNFunction(torch.autograd.Function):
    """x + (act(x Wg + bg) * (x Wu + bu)) Wd + bd as one autograd node."""

    @staticmethod
    def forward(ctx, x, act, residual, Wg, Wu, Wd, bg, bu, bd):
        H, (Zg, Zu) = gated_gemm_train(x, Wg, Wu, bg, bu, act=act)
        y = gemm_residual(H, Wd, x if residual else None, bd)
        ctx.act, ctx.residual = act, residual
        ctx.save_for_backward(x, Wg, Wu, Wd, Zg, Zu, H)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, Wg, Wu, Wd, Zg, Zu, H = ctx.saved_tensors
        need = ctx.needs_input_grad
        dy = _rows16(dy.to(x.dtype))
        down = gemm_residual_backward(H, Wd, dy, want_dB=need[5], want_dbias=need[8], grad_dtype=Wd.dtype)
        up = gated_gemm_backward(x, Wg, Wu, (Zg, Zu), down.dA, act=ctx.act, want_dA=need[0],
                                 want_dB=need[3] or need[4], want_dbias=need[6] or need[7], grad_dtype=Wg.dtype)
        dx = up.dA
        if need[0] and ctx.residual:
            dx = dx + dy
        return dx, None, None, up.dBg, up.dBu, down.dB, up.dbias_g, up.dbias_u, down.dbias


class GatedFFN(torch.nn.Module):
    """The gated feed-forward block ``y = x + (act(x Wg + bg) * (x Wu + bu)) Wd + bd``.

    Weights in the x @ W orientation.  ``residual=False`` leaves out the
    ``x +``, ``bias=False`` (the default) the biases.  x is ``[..., D]``.
    """

    def __init__(self, D: int, H: int, act="silu", bias: bool = False, residual: bool = True, device="cuda",
                 dtype=torch.bfloat16):
        super().__init__()
        _act(act)
        self.act, self.residual, self.D, self.H = act, residual, D, H

        def param(*shape, std=0.0):
            p = torch.nn.Parameter(torch.zeros(*shape, device=device, dtype=dtype))
            if std:
                torch.nn.init.normal_(p, std=std)
            return p

        self.Wg, self.Wu = param(D, H, std=D ** -0.5), param(D, H, std=D ** -0.5)
        self.Wd = param(H, D, std=H ** -0.5)
        self.bg, self.bu, self.bd = (param(H), param(H), param(D)) if bias else (None, None, None)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        shape = x.shape
        x2 = _rows16(x.reshape(-1, self.D))
        Wg, Wu, Wd = _rows16(self.Wg), _rows16(self.Wu), _rows16(self.Wd)
        if torch.is_grad_enabled() and (x.requires_grad or any(p.requires_grad for p in self.parameters())):
            y = _GatedFFNFunction.apply(x2, self.act, self.residual, Wg, Wu, Wd, self.bg, self.bu, self.bd)
        else:
            h = gated_gemm(x2, Wg, Wu, self.bg, self.bu, act=self.act)
            y = gemm_residual(h, Wd, x2 if self.residual else None, self.bd)
        return y.reshape(shape)
