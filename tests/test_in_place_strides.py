"""The gated backward calls write da over a row by row: a's own address with
another stride is refused (rows would be overwritten before they are read).  The
pointers are fake, no call gets to the device."""
import ctypes

import pytest

from helpers import build_lib

P, Q, NULL = ctypes.c_void_p(4096), ctypes.c_void_p(1 << 20), None


@pytest.fixture(scope="module")
def ops():
    build_lib()
    from grouped_gemm_top_gb300 import ops
    return ops


def grouped(ops, **k):
    a = dict(dh=P, lddh=24, a=P, lda=56, x=P, ldx=64, w=P, ldw=48, gsw=64 * 48, act=3, o=P, r=P, G=4, M=16, f=24, d=64, da=P,
             ldda=56, dx=P, lddx=64, dw=P, dwt=0, lddw=48, gsdw=64 * 48)
    a.update(k)
    return ops.lib.grouped_ffn_bwd(*a.values(), NULL, NULL)


def dense(ops, **k):
    a = dict(dh=P, lddh=24, a=P, lda=56, x=P, ldx=64, w=P, ldw=48, act=3, M=16, f=24, d=64, da=P, ldda=56, dx=P, lddx=64, dw=P,
             dwt=0, lddw=48)
    a.update(k)
    return ops.lib.gated_ffn_bwd(*a.values(), NULL, NULL)


@pytest.mark.parametrize("call", [grouped, dense])
def test_the_same_stride(ops, call):
    for k in (dict(ldda=48), dict(ldda=64), dict(lda=48)):
        assert call(ops, **k) == ops.MOE_ERR_INVALID_ARG, k
    for k in (dict(), dict(da=Q, ldda=48), dict(M=1, ldda=48), dict(lda=48, ldda=48)):      # a row has no stride
        assert call(ops, **k) == ops.MOE_ERR_NOT_INITIALIZED, k
