"""Host-side checks of the feed-forward entry points that need no GPU: every
invalid or unsupported request is refused with its documented status before
any device call (fake pointers, never dereferenced); a request that passes
every check reaches the device query, which fails here."""
import ctypes

import pytest

import mlp_megakernel_amd as mk

INV, UNS, DEV = mk.ERR_INVALID_ARGUMENT, mk.ERR_UNSUPPORTED, mk.ERR_DEVICE
P = 0x100000  # distinct 16-byte aligned fake addresses, 1 MB apart
M, N, K = 8, 64, 48


@pytest.fixture(autouse=True)
def _without_gpu():
    import torch
    if torch.cuda.is_available():
        pytest.skip("the accepting cases would launch on fake pointers")


def residual(**kw):
    a = dict(A=P, lda=K, B=2 * P, ldb=N, bias=None, R=3 * P, ldr=N, Z=None, ldz=0, Y=4 * P, ldy=N, M=M, N=N, K=K,
             i=mk.BF16, o=mk.BF16, act=mk.ACT_SILU, ws=None, n=0)
    a.update(kw)
    return mk.load_library().coalesce_gemm_residual(*[a[k] for k in (
        "A", "lda", "B", "ldb", "bias", "R", "ldr", "Z", "ldz", "Y", "ldy", "M", "N", "K", "i", "o", "act", "ws", "n")],
        None)


def gated(**kw):
    a = dict(A=P, lda=K, Bg=2 * P, Bu=3 * P, ldb=N, bg=None, bu=None, Zg=None, Zu=None, ldz=N, Y=4 * P, ldy=N,
             M=M, N=N, K=K, i=mk.F16, o=mk.F16, act=mk.ACT_SILU, ws=None, n=0)
    a.update(kw)
    return mk.load_library().coalesce_gated_gemm(*[a[k] for k in (
        "A", "lda", "Bg", "Bu", "ldb", "bg", "bu", "Zg", "Zu", "ldz", "Y", "ldy", "M", "N", "K", "i", "o",
        "act", "ws", "n")], None)


def residual_bwd(**kw):
    a = dict(A=P, lda=K, B=2 * P, ldb=N, Z=3 * P, ldz=N, dY=4 * P, ldd=N, dA=5 * P, ldda=K, dB=6 * P, lddb=N, db=None,
             M=M, N=N, K=K, i=mk.BF16, d=mk.BF16, g=mk.F32, act=mk.ACT_GELU_ERF, ws=16 * P, n=1 << 30)
    a.update(kw)
    return mk.load_library().coalesce_gemm_residual_backward(*[a[k] for k in (
        "A", "lda", "B", "ldb", "Z", "ldz", "dY", "ldd", "dA", "ldda", "dB", "lddb", "db", "M", "N", "K", "i", "d", "g",
        "act", "ws", "n")], None)


def gated_bwd(**kw):
    a = dict(A=P, lda=K, Bg=2 * P, Bu=3 * P, ldb=N, Zg=4 * P, Zu=5 * P, ldz=N, dY=6 * P, ldd=N, dA=7 * P,
             ldda=K, dBg=8 * P, dBu=9 * P, lddb=N, bg=None, bu=None, M=M, N=N, K=K, i=mk.BF16, d=mk.BF16,
             g=mk.F32, act=mk.ACT_SILU, ws=16 * P, n=1 << 30)
    a.update(kw)
    return mk.load_library().coalesce_gated_gemm_backward(*[a[k] for k in (
        "A", "lda", "Bg", "Bu", "ldb", "Zg", "Zu", "ldz", "dY", "ldd", "dA", "ldda", "dBg", "dBu", "lddb", "bg", "bu", "M", "N", "K", "i", "d", "g", "act", "ws", "n")], None)


COMMON = [(dict(M=-1), INV), (dict(N=-1), INV), (dict(K=-5), INV), (dict(i=9), INV), (dict(act=5), INV),
          (dict(act=-1), INV), (dict(i=mk.F32), UNS), (dict(M=(1 << 31) - 200), UNS),
          (dict(M=1 << 21, N=1 << 21, ldy=1 << 21, ldz=1 << 21, ldd=1 << 21, ldb=1 << 21), UNS),
          (dict(A=None), INV), (dict(A=P + 8), UNS), (dict(lda=K - 1), INV), (dict(lda=K + 4), UNS),
          (dict(lda=1 << 23), UNS)]
FORWARD = [(dict(o=mk.F32 + 7), INV), (dict(Y=None), INV), (dict(Y=4 * P + 4), UNS), (dict(ldy=N - 8), INV),
           (dict(ldy=N + 4), UNS), (dict(Y=P + 16), INV)]


@pytest.mark.parametrize("kw,status", COMMON + FORWARD + [
    (dict(o=mk.F16), UNS), (dict(B=None), INV), (dict(B=2 * P + 2), UNS), (dict(ldb=N - 1), INV),
    (dict(ldr=N - 1), INV), (dict(R=3 * P + 4), UNS), (dict(R=4 * P, ldr=N + 8), INV), (dict(R=4 * P + 16), INV),
    (dict(Z=4 * P, ldz=N), INV), (dict(Z=5 * P, ldz=N - 8), INV), (dict(bias=6 * P + 2), UNS),
    (dict(bias=4 * P), INV), (dict(Z=2 * P + 16, ldz=N), INV)])
def test_residual_refuses(kw, status):
    assert residual(**kw) == status
    assert len(mk.load_library().coalesce_last_error()) > 0


@pytest.mark.parametrize("kw,status", COMMON + FORWARD + [
    (dict(o=mk.BF16), UNS), (dict(Bg=None), INV), (dict(Bu=None), INV), (dict(Bu=3 * P + 4), UNS),
    (dict(ldb=N - 8), INV), (dict(Zg=5 * P), INV), (dict(Zu=5 * P), INV), (dict(Zg=5 * P, Zu=5 * P), INV),
    (dict(Zg=5 * P, Zu=5 * P + 16), INV), (dict(Zg=5 * P, Zu=4 * P), INV), (dict(bu=5 * P + 2), UNS)])
def test_gated_refuses(kw, status):
    assert gated(**kw) == status


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(d=9), INV), (dict(d=mk.F16), UNS), (dict(g=mk.F16), UNS), (dict(g=-1), INV), (dict(B=None), INV),
    (dict(Z=None), INV), (dict(Z=3 * P + 2), UNS), (dict(dY=None), INV), (dict(ldd=N - 1), INV),
    (dict(dA=5 * P + 4), UNS), (dict(ldda=K - 1), INV), (dict(dA=P), INV), (dict(dB=4 * P), INV),
    (dict(dB=5 * P), INV), (dict(lddb=N - 1), INV), (dict(db=6 * P), INV), (dict(db=7 * P + 4), UNS)])
def test_residual_backward_refuses(kw, status):
    assert residual_bwd(**kw) == status


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(d=mk.F16), UNS), (dict(g=mk.F16), UNS), (dict(Bu=None), INV), (dict(Zu=None), INV), (dict(dY=None), INV),
    (dict(dBu=8 * P), INV), (dict(dBu=8 * P + 16), INV), (dict(dBg=6 * P), INV), (dict(dA=4 * P), INV),
    (dict(bg=10 * P, bu=10 * P), INV), (dict(lddb=N - 4), INV)])
def test_gated_backward_refuses(kw, status):
    assert gated_bwd(**kw) == status


def test_accepted_requests_reach_the_device():
    assert residual() == DEV and gated() == DEV and residual_bwd() == DEV and gated_bwd() == DEV
    assert residual(R=None, ldr=0) == DEV and residual(R=4 * P) == DEV           # none, in place
    assert residual(i=mk.F16, o=mk.F32) == DEV and gated(Zg=5 * P, Zu=6 * P) == DEV
    # halves of one matrix: weights, their gradients, the stored pre-activations
    assert gated(Bu=2 * P + 2 * N, ldb=2 * N, Zg=5 * P, Zu=5 * P + 2 * N, ldz=2 * N) == DEV
    assert gated_bwd(dBu=8 * P + 4 * N, lddb=2 * N) == DEV
    # unwanted gradients need no matching inputs
    assert residual_bwd(dA=None, B=None) == DEV and residual_bwd(dB=None, A=None) == DEV
    assert residual_bwd(act=mk.ACT_NONE, Z=None) == DEV


def test_empty_requests_need_no_device():
    assert residual(M=0, A=None, Y=None, R=None) == mk.OK and gated(N=0, Y=None) == mk.OK
    assert residual_bwd(dA=None, dB=None) == mk.OK and gated_bwd(dA=None, dBg=None, dBu=None) == mk.OK
    assert residual_bwd(M=0, dB=None) == mk.OK
    lib = mk.load_library()
    for name in ("gemm_residual", "gated_gemm"):
        assert getattr(lib, "coalesce_%s_workspace_size" % name)(-1, 4, 4) == 0
        assert getattr(lib, "coalesce_%s_backward_workspace_size" % name)(4, 4, 1 << 40) == 0


def test_other_entry_points_refuse_silu():
    lib = mk.load_library()
    assert lib.coalesce_gemm_bias_act(P, 64, 2 * P, 64, None, 4 * P, 64, 8, 64, 64, mk.F32, mk.F32, mk.ACT_SILU,
                                      None) == INV
    assert lib.coalesce_activation(P, 64, 4 * P, 64, 4, 64, mk.F32, mk.ACT_SILU, None) == INV


def clip(src, dst, numel, dts, count=None, norm_type=mk.NORM_2, max_norm=1.0, norm=64 * P, ws=65 * P, n=1 << 20):
    def arr(ct, v):
        return None if v is None else ctypes.cast((ct * max(1, len(v)))(*v), ctypes.c_void_p)
    count = len(numel) if count is None else count
    return mk.load_library().coalesce_clip_grad_norm(
        arr(ctypes.c_void_p, src), arr(ctypes.c_void_p, dst), arr(ctypes.c_int64, numel), arr(ctypes.c_int32, dts),
        count, norm_type, max_norm, norm, ws, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(count=-1), INV), (dict(norm_type=2), INV), (dict(norm=None), INV), (dict(norm=64 * P + 2), UNS),
    (dict(max_norm=-1.0), INV), (dict(max_norm=float("nan")), INV), (dict(src=None), INV), (dict(dst=None), INV),
    (dict(numel=None, count=2), INV), (dict(dts=None), INV), (dict(numel=[4, -1]), INV), (dict(dts=[0, 3]), INV),
    (dict(src=[P, None]), INV), (dict(dst=[None, P]), INV), (dict(src=[P + 2, 2 * P]), UNS),
    (dict(dst=[P, 2 * P + 1]), UNS), (dict(numel=[1 << 47, 1 << 48]), UNS)])
def test_clip_refuses(kw, status):
    a = dict(src=[P, 2 * P], dst=[P, 2 * P], numel=[100, 100], dts=[mk.F32, mk.BF16])
    a.update(kw)
    assert clip(**a) == status


def test_clip_accepted_reaches_the_device():
    assert clip([P, 2 * P], [P, 3 * P], [100, 100], [mk.F32, mk.BF16]) == DEV
    assert clip([], [], [], []) == DEV


def test_binding_refuses():
    import torch
    a = torch.zeros(4, 8, dtype=torch.bfloat16)
    for call in (lambda: mk.gated_gemm(a, a, a), lambda: mk.gemm_residual(a, a),
                 lambda: mk.gemm_residual_backward(a, a, a), lambda: mk.gated_gemm_backward(a, a, a, (a, a), a)):
        with pytest.raises(ValueError):
            call()
    for grads, out in (([a], None), ([None], None), ([1.0], None), ([], [a]), ([a], [a]), ([a, a], [a])):
        with pytest.raises(ValueError):
            mk.clip_grad_norm(grads, 1.0, out=out)
    with pytest.raises(TypeError):
        mk.clip_grad_norm(3, 1.0)
    with pytest.raises(ValueError):
        mk.GatedFFN(8, 8, act="swish?", device="cpu")
