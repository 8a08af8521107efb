"""Host-side checks of the entry points around the feed-forward products that
need no GPU: every invalid or unsupported request is refused with its documented
status before any device call (fake pointers, never dereferenced); a request
that passes every check reaches the device query, which fails here.  And the
reference generator gives the published vectors."""
import numpy as np
import pytest

import block_reference as ref
import mlp_megakernel_amd as mk

INV, UNS, DEV = mk.ERR_INVALID_ARGUMENT, mk.ERR_UNSUPPORTED, mk.ERR_DEVICE
P = 0x100000  # distinct 16-byte aligned fake addresses, 1 MB apart
M, N = 8, 64


@pytest.fixture(autouse=True)
def _without_gpu():
    import torch
    if torch.cuda.is_available():
        pytest.skip("the accepting cases would launch on fake pointers")


def call(name, defaults, kw):
    assert set(kw) <= set(defaults)
    a = {**defaults, **kw}
    return getattr(mk.load_library(), name)(*a.values(), None)


NORM = dict(X=P, ldx=N, R=2 * P, ldr=N, S=3 * P, lds=N, weight=4 * P, bias=5 * P, Y=6 * P, ldy=N, mean=7 * P,
            rstd=8 * P, M=M, N=N, dt=mk.BF16, sdt=mk.BF16, wdt=mk.BF16, eps=1e-5, p=0.1, seed=1, offset=0, dev=None)
BACK = dict(S=P, lds=N, weight=2 * P, mean=3 * P, rstd=4 * P, dY=5 * P, ldy=N, dS=6 * P, ldg=N, dX=7 * P, ldx=N,
            dB=8 * P, ldb=N, dweight=9 * P, dbias=10 * P, M=M, N=N, dt=mk.F16, sdt=mk.F32, wdt=mk.F16, gdt=mk.F32,
            p=0.1, seed=1, offset=0, dev=None, ws=16 * P, n=1 << 30)
DROP = dict(X=P, ldx=N, R=2 * P, ldr=N, Y=3 * P, ldy=N, M=M, N=N, dt=mk.BF16, odt=mk.F32, p=0.1, seed=1, offset=0,
            dev=None)
COMMON = [(dict(M=-1), INV), (dict(N=-1), INV), (dict(M=(1 << 31) - 200), UNS), (dict(M=1 << 21, N=1 << 21), UNS),
          (dict(dt=9), INV), (dict(p=-0.1), INV), (dict(p=1.01), INV), (dict(p=float("nan")), INV),
          (dict(dev=12 * P + 4), UNS)]


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(sdt=mk.F16), UNS), (dict(wdt=mk.F16), UNS), (dict(dt=mk.F32), UNS), (dict(wdt=-1), INV),
    (dict(X=None), INV), (dict(X=P + 8), UNS), (dict(ldx=N - 8), INV), (dict(ldx=N + 4), UNS), (dict(ldx=1 << 23), UNS),
    (dict(Y=None), INV), (dict(Y=P), INV), (dict(Y=3 * P + 16), INV), (dict(ldy=N - 1), INV), (dict(S=3 * P + 2), UNS),
    (dict(S=2 * P, lds=N + 8), INV), (dict(S=2 * P + 16), INV), (dict(R=None), INV), (dict(R=None, S=None), INV),
    (dict(R=2 * P + 4), UNS), (dict(ldr=N - 8), INV), (dict(weight=4 * P + 2), UNS), (dict(bias=6 * P), INV),
    (dict(mean=7 * P + 2), UNS), (dict(rstd=7 * P), INV), (dict(mean=6 * P + 4), INV), (dict(eps=-1e-9), INV),
    (dict(eps=float("inf")), INV), (dict(eps=float("nan")), INV), (dict(dev=6 * P), INV)])
def test_norm_refuses(kw, status):
    assert call("coalesce_layer_norm", NORM, kw) == status
    assert len(mk.load_library().coalesce_last_error()) > 0


@pytest.mark.parametrize("kw,status", [
    (dict(), DEV), (dict(S=2 * P), DEV), (dict(S=None), DEV), (dict(R=None, S=None, p=0.0), DEV),
    (dict(sdt=mk.F32, wdt=mk.F32), DEV), (dict(mean=None, rstd=None, weight=None, bias=None), DEV),
    (dict(M=0), 0), (dict(N=0), 0), (dict(M=0, X=None, Y=None), 0), (dict(M=0, R=None), 0),
    (dict(p=1.0, dev=12 * P), DEV), (dict(dev=6 * P, p=0.0), DEV)])
def test_norm_accepts(kw, status):
    assert call("coalesce_layer_norm", NORM, kw) == status


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(sdt=mk.BF16), UNS), (dict(wdt=mk.BF16), UNS), (dict(gdt=mk.BF16), UNS), (dict(gdt=7), INV),
    (dict(S=None), INV), (dict(dY=None), INV), (dict(mean=None), INV), (dict(rstd=None), INV),
    (dict(rstd=4 * P + 1), UNS),
    (dict(dS=7 * P, ldg=N + 8), INV), (dict(dX=7 * P + 8), UNS), (dict(dX=5 * P), INV), (dict(dB=7 * P + 64), INV),
    (dict(dweight=9 * P + 4), UNS), (dict(dbias=9 * P), INV), (dict(dweight=2 * P), INV), (dict(ldb=N - 8), INV),
    (dict(M=0, N=1 << 28), UNS)])
def test_norm_backward_refuses(kw, status):
    assert call("coalesce_layer_norm_backward", BACK, kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(), DEV), (dict(dS=7 * P), DEV), (dict(dS=None, dX=None, dB=None), DEV), (dict(dweight=None, dbias=None), DEV),
    (dict(dX=None, dB=None, dweight=None, dbias=None), 0), (dict(N=0), 0), (dict(M=0, dweight=None, dbias=None), 0),
    (dict(M=0, S=None, dY=None, mean=None, rstd=None), DEV), (dict(weight=None), DEV)])
def test_norm_backward_accepts(kw, status):
    assert call("coalesce_layer_norm_backward", BACK, kw) == status
    assert mk.load_library().coalesce_layer_norm_backward_workspace_size(8, 64) == 0  # (no device here)


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(odt=mk.F16), UNS), (dict(dt=mk.F32, odt=mk.BF16), UNS), (dict(X=None), INV), (dict(Y=None), INV),
    (dict(X=P + 4), UNS), (dict(Y=P), INV), (dict(X=3 * P), INV), (dict(R=3 * P, ldr=N + 4), INV),
    (dict(R=3 * P + 16), INV), (dict(ldr=N - 4), INV), (dict(ldy=N + 2), UNS), (dict(dev=3 * P), INV)])
def test_dropout_refuses(kw, status):
    assert call("coalesce_dropout", DROP, kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(), DEV), (dict(R=None), DEV), (dict(R=3 * P), DEV), (dict(odt=mk.BF16, X=3 * P), DEV), (dict(p=0.0), DEV),
    (dict(M=0, X=None), 0), (dict(N=0), 0)])
def test_dropout_accepts(kw, status):
    assert call("coalesce_dropout", DROP, kw) == status


@pytest.mark.parametrize("counter,key,want", [
    ([0, 0, 0, 0], [0, 0], [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
    ([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
    ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0],
     [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1])])
def test_generator_gives_the_published_vectors(counter, key, want):
    got = ref.philox([np.array([c]) for c in counter], key)
    assert [int(g[0]) for g in got] == want


# ---------------------------------------------------------------------------
# 8-bit operands
# ---------------------------------------------------------------------------

K = 48
INT8 = dict(A=P, lda=K, B=2 * P, ldb=K, sa=3 * P, sb=4 * P, bias=5 * P, R=6 * P, ldr=N, Y=7 * P, ldy=N, M=M, N=N, K=K,
            odt=mk.BF16, act=mk.ACT_GELU_ERF, ws=16 * P, n=1 << 30)
GATED8 = dict(A=P, lda=K, Bg=2 * P, Bu=3 * P, ldb=K, sa=4 * P, sg=5 * P, su=6 * P, bg=7 * P, bu=8 * P, Y=9 * P, ldy=N,
              M=M, N=N, K=K, odt=mk.F32, act=mk.ACT_SILU, ws=16 * P, n=1 << 30)
QUANT = dict(X=P, ldx=N, Q=2 * P, ldq=N, scale=3 * P, M=N, N=N, dt=mk.BF16)
BOTH = [(dict(M=-1), INV), (dict(N=-2), INV), (dict(K=-1), INV), (dict(K=131072, lda=131072, ldb=131072), UNS),
        (dict(M=(1 << 31) - 200), UNS), (dict(M=1 << 21, N=1 << 21), UNS), (dict(odt=5), INV), (dict(act=9), INV),
        (dict(A=None), INV), (dict(A=P + 8), UNS), (dict(lda=K - 16), INV), (dict(lda=K + 8), UNS),
        (dict(lda=1 << 23), UNS), (dict(ldb=K - 16), INV), (dict(sa=None), INV), (dict(sa=3 * P + 2), UNS),
        (dict(Y=None), INV), (dict(ldy=N - 8), INV), (dict(Y=P + 16), INV)]


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(B=None), INV), (dict(B=2 * P + 4), UNS), (dict(sb=None), INV), (dict(sb=4 * P + 8), UNS),
    (dict(bias=5 * P + 4), UNS), (dict(R=7 * P, ldr=N + 8), INV), (dict(R=7 * P + 32), INV), (dict(R=6 * P + 2), UNS),
    (dict(bias=7 * P), INV), (dict(sb=7 * P), INV)])
def test_int8_refuses(kw, status):
    assert call("coalesce_gemm_int8", INT8, kw) == status


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(Bg=None), INV), (dict(Bu=None), INV), (dict(Bu=3 * P + 4), UNS), (dict(sg=None), INV), (dict(su=None), INV),
    (dict(su=6 * P + 4), UNS), (dict(bu=8 * P + 4), UNS), (dict(bu=9 * P), INV)])
def test_gated_int8_refuses(kw, status):
    assert call("coalesce_gated_gemm_int8", GATED8, kw) == status


@pytest.mark.parametrize("kw", [dict(M=-1), dict(dt=4)])
def test_quantize_refuses_invalid(kw):
    for name in ("coalesce_quantize_rows", "coalesce_quantize_columns"):
        assert call(name, QUANT, kw) == INV


@pytest.mark.parametrize("kw,status", [
    (dict(X=None), INV), (dict(X=P + 2), UNS), (dict(Q=None), INV), (dict(Q=2 * P + 8), UNS), (dict(ldq=N - 16), INV),
    (dict(ldq=N + 8), UNS), (dict(ldx=N - 8), INV), (dict(scale=None), INV), (dict(scale=3 * P + 2), UNS),
    (dict(Q=P), INV), (dict(scale=2 * P), INV), (dict(M=(1 << 31) - 1), UNS), (dict(), DEV), (dict(M=0, N=0), 0)])
def test_quantize_checks(kw, status):
    for name in ("coalesce_quantize_rows", "coalesce_quantize_columns"):
        assert call(name, QUANT, kw) == status


def test_int8_accepts():
    for name, defaults in (("coalesce_gemm_int8", INT8), ("coalesce_gated_gemm_int8", GATED8)):
        assert call(name, defaults, {}) == DEV
        assert call(name, defaults, dict(K=131071, lda=131072, ldb=131072, N=8)) == DEV
        assert call(name, defaults, dict(K=0, A=None)) == DEV
        assert call(name, defaults, dict(M=0, A=None, Y=None)) == 0
    assert call("coalesce_gemm_int8", INT8, dict(R=7 * P, sa=3 * P + 4)) == DEV
    assert call("coalesce_quantize_rows", QUANT, dict(scale=3 * P + 4)) == DEV
    assert call("coalesce_quantize_rows", QUANT, dict(M=0)) == 0
    assert call("coalesce_quantize_rows", QUANT, dict(N=0, X=None, Q=None)) == DEV
    assert mk.load_library().coalesce_gemm_int8_workspace_size(8, 64, 131072) == 0
