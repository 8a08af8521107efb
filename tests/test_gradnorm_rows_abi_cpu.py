"""Host-side checks of the gradient-norm entry points over matrices whose rows lie
apart: refused with the documented status before any device call; a list that
passes every check reaches the device query, which fails here."""
import ctypes

import pytest

import mlp_megakernel_amd as mk

INV, UNS, DEV = mk.ERR_INVALID_ARGUMENT, mk.ERR_UNSUPPORTED, mk.ERR_DEVICE
P = 0x100000  # fake addresses, never dereferenced


@pytest.fixture(autouse=True)
def _without_gpu():
    import torch
    if torch.cuda.is_available():
        pytest.skip("the accepting cases would launch on fake pointers")


def arr(ct, v):
    return None if v is None else ctypes.cast((ct * max(1, len(v)))(*v), ctypes.c_void_p)


def clip(src=(P, 2 * P), dst=(P, 3 * P), numel=(120, 100), cols=(12, 0), ld=(16, 0), ldo=(16, 0),
         dts=(mk.F32, mk.BF16), max_norm=1.0):
    i64 = ctypes.c_int64
    return mk.load_library().coalesce_clip_grad_norm_rows(
        arr(ctypes.c_void_p, src), arr(ctypes.c_void_p, dst), arr(i64, numel), arr(i64, cols), arr(i64, ld), arr(i64, ldo),
        arr(ctypes.c_int32, dts), len(numel), mk.NORM_2, max_norm, 64 * P, 65 * P, 1 << 20, None)


@pytest.mark.parametrize("kw,status", [
    (dict(cols=(-12, 0)), INV), (dict(cols=(13, 0)), INV), (dict(ld=(11, 0)), INV), (dict(ldo=(11, 0)), INV),
    (dict(ldo=(20, 0)), INV), (dict(ld=None), INV), (dict(ldo=None), INV), (dict(ld=(1 << 45, 0), ldo=(1 << 45, 0)), UNS),
    (dict(max_norm=-1.0), INV), (dict(dst=None), INV), (dict(src=(P, None)), INV)])
def test_refuses(kw, status):
    assert clip(**kw) == status


def test_accepted_reaches_the_device():
    assert clip() == DEV and clip(dst=(4 * P, 3 * P), ldo=(20, 0)) == DEV
    assert clip(cols=None, ld=None, ldo=None) == DEV and clip(numel=(0, 100), cols=(12, 0)) == DEV
    i64 = ctypes.c_int64
    assert mk.load_library().coalesce_grad_norm_rows(
        arr(ctypes.c_void_p, [P]), arr(i64, [24]), arr(i64, [6]), arr(i64, [8]), arr(ctypes.c_int32, [mk.F16]), 1, mk.NORM_INF,
        64 * P, 65 * P, 1 << 20, None) == DEV


def test_workspace_size_of_invalid_lists():
    i64 = ctypes.c_int64
    f = mk.load_library().coalesce_grad_norm_rows_workspace_size
    for numel, cols in (([10], [3]), ([10], [-5]), ([-1], [1])):
        assert f(arr(i64, numel), arr(i64, cols), arr(ctypes.c_int32, [0]), 1) == 0
    assert f(None, None, None, 0) == 0
