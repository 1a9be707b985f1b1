"""Host-side checks of the grouped bf16 products' and the distillation loss's C
entry points: every call here is refused (or has nothing to do) before any device
work, the pointers are fake."""
import ctypes

import pytest

from helpers import build_lib

P, ODD, NULL = ctypes.c_void_p(4096), ctypes.c_void_p(4097), None


@pytest.fixture(scope="module")
def ops():
    build_lib()
    from grouped_gemm_top_gb300 import ops
    return ops


def lin_fwd(ops, **k):
    a = dict(x=P, ldx=64, w=P, ldw=48, gsw=64 * 48, o=P, r=P, G=4, M=16, N=48, K=64, y=P, ldy=48)
    a.update(k)
    return ops.lib.grouped_linear_fwd(*a.values(), NULL, NULL)


def lin_bwd(ops, **k):
    a = dict(dy=P, lddy=48, x=P, ldx=64, w=P, ldw=48, gsw=64 * 48, o=P, r=P, G=4, M=16, N=48, K=64, dx=P, lddx=64, dw=P,
             dwt=0, lddw=48, gsdw=64 * 48)
    a.update(k)
    return ops.lib.grouped_linear_bwd(*a.values(), NULL, NULL)


def ffn_fwd(ops, **k):
    a = dict(x=P, ldx=64, w=P, ldw=48, gsw=64 * 48, act=3, o=P, r=P, G=4, M=16, f=24, d=64, h=P, ldh=24, a=P, lda=48)
    a.update(k)
    return ops.lib.grouped_ffn_fwd(*a.values(), NULL, NULL)


def ffn_bwd(ops, **k):
    a = dict(dh=P, lddh=24, a=P, lda=48, x=P, ldx=64, w=P, ldw=48, gsw=64 * 48, act=3, o=P, r=P, G=4, M=16, f=24, d=64, da=P,
             ldda=48, dx=P, lddx=64, dw=P, dwt=0, lddw=48, gsdw=64 * 48)
    a.update(k)
    return ops.lib.grouped_ffn_bwd(*a.values(), NULL, NULL)


def test_grouped_linear(ops):
    inv, uns, ali = ops.MOE_ERR_INVALID_ARG, ops.MOE_ERR_UNSUPPORTED, ops.MOE_ERR_ALIGNMENT
    for k in (dict(M=-1), dict(N=0), dict(K=0), dict(G=0), dict(x=NULL), dict(w=NULL), dict(y=NULL), dict(o=NULL),
              dict(ldx=63), dict(ldw=47), dict(ldy=47), dict(gsw=64 * 48 - 1), dict(gsw=0)):
        assert lin_fwd(ops, **k) == inv, k
    for k in (dict(x=ODD), dict(w=ODD), dict(y=ODD), dict(o=ODD), dict(r=ODD), dict(ldx=68), dict(gsw=64 * 48 + 4)):
        assert lin_fwd(ops, **k) == ali, k
    assert lin_fwd(ops, M=1 << 31) == uns and lin_fwd(ops, G=65537) == uns
    assert lin_fwd(ops, M=0, x=NULL, y=NULL, o=NULL) == ops.MOE_OK
    assert lin_fwd(ops, M=1, ldx=67, ldy=51, G=1, gsw=0) == ops.MOE_ERR_NOT_INITIALIZED      # strides of one row, one group


def test_grouped_linear_backward(ops):
    inv, ali = ops.MOE_ERR_INVALID_ARG, ops.MOE_ERR_ALIGNMENT
    for k in (dict(M=-1), dict(N=0), dict(G=0), dict(dy=NULL), dict(x=NULL), dict(w=NULL), dict(o=NULL), dict(dwt=2),
              dict(dx=NULL, dw=NULL), dict(lddy=47), dict(lddx=63), dict(lddw=47), dict(gsdw=5)):
        assert lin_bwd(ops, **k) == inv, k
    for k in (dict(dy=ODD), dict(x=ODD), dict(w=ODD), dict(dx=ODD), dict(dw=ODD), dict(o=ODD), dict(gsdw=64 * 48 + 4)):
        assert lin_bwd(ops, **k) == ali, k
    # what is not asked for is not looked at
    assert lin_bwd(ops, dx=NULL, w=NULL, ldw=0, gsw=0) == ops.MOE_ERR_NOT_INITIALIZED
    assert lin_bwd(ops, dw=NULL, x=NULL, ldx=0, lddw=0) == ops.MOE_ERR_NOT_INITIALIZED


def test_grouped_gated(ops):
    inv, uns, ali = ops.MOE_ERR_INVALID_ARG, ops.MOE_ERR_UNSUPPORTED, ops.MOE_ERR_ALIGNMENT
    for k in (dict(act=4), dict(act=-1), dict(f=0), dict(d=0), dict(x=NULL), dict(h=NULL), dict(o=NULL), dict(ldw=47),
              dict(ldh=23), dict(lda=47), dict(gsw=1)):
        assert ffn_fwd(ops, **k) == inv, k
    assert ffn_fwd(ops, f=20, ldw=40, gsw=64 * 40) == uns
    for k in (dict(x=ODD), dict(w=ODD), dict(h=ODD), dict(a=ODD), dict(r=ODD)):
        assert ffn_fwd(ops, **k) == ali, k
    assert ffn_fwd(ops, M=0) == ops.MOE_OK
    for k in (dict(act=9), dict(dwt=5), dict(dh=NULL), dict(a=NULL), dict(da=NULL), dict(o=NULL), dict(ldda=47), dict(lddx=1)):
        assert ffn_bwd(ops, **k) == inv, k
    assert ffn_bwd(ops, f=20, lddw=40, gsdw=64 * 40) == uns
    for k in (dict(dh=ODD), dict(a=ODD), dict(da=ODD), dict(x=ODD), dict(dw=ODD)):
        assert ffn_bwd(ops, **k) == ali, k


def args(**k):
    a = dict(x=P, xt=0, ldx=100, idx=P, ldi=8, t=P, tt=1, ldt=8, lse=P, tau=1.0, M=4, V=100, k=8)
    a.update(k)
    return a


def distill(ops, which, **k):
    extra = {n: k.pop(n) for n in ("loss", "stats", "dloss", "dx", "lddx") if n in k}
    a = list(args(**k).values())
    e = dict(loss=P, stats=P, dloss=P, dx=P, lddx=100)
    e.update(extra)
    if which == "fwd":
        return ops.lib.distill_loss_fwd(*a, e["loss"], e["stats"], NULL, NULL)
    if which == "bwd":
        return ops.lib.distill_loss_bwd(e["dloss"], *a[:8], e["stats"], *a[8:], e["dx"], e["lddx"], NULL, NULL)
    return ops.lib.distill_loss(e["dloss"], *a, e["loss"], e["dx"], e["lddx"], NULL, NULL)


@pytest.mark.parametrize("which", ["fwd", "bwd", "both"])
def test_distillation(ops, which):
    inv, uns, ali = ops.MOE_ERR_INVALID_ARG, ops.MOE_ERR_UNSUPPORTED, ops.MOE_ERR_ALIGNMENT
    for k in (dict(x=NULL), dict(idx=NULL), dict(t=NULL), dict(xt=2), dict(tt=-1), dict(M=-1), dict(V=0), dict(k=0),
              dict(ldx=99), dict(ldi=7), dict(ldt=7), dict(tau=0.0), dict(tau=-1.0), dict(tau=float("nan")),
              dict(tau=float("inf"))):
        assert distill(ops, which, **k) == inv, k
    for k in (dict(M=1 << 31), dict(k=1025, ldi=1025, ldt=1025), dict(V=720883, ldx=800000, lddx=800000),
              dict(V=360443, ldx=800000, lddx=800000, xt=1)):
        assert distill(ops, which, **k) == uns, k
    two = ctypes.c_void_p(4098)
    for k in (dict(x=ODD), dict(x=two, xt=1), dict(idx=two), dict(t=two), dict(lse=two)):
        assert distill(ops, which, **k) == ali, k
    assert distill(ops, which, M=0, x=NULL, idx=NULL, t=NULL, dx=NULL, dloss=NULL) == ops.MOE_OK
    if which != "fwd":
        for k in (dict(dloss=NULL), dict(dx=NULL), dict(lddx=99), dict(lddx=104)):      # the last: in place, another stride
            assert distill(ops, which, **k) == inv, k
        assert distill(ops, which, dx=ODD) == ali and distill(ops, which, dx=ctypes.c_void_p(8192), dloss=two) == ali
    if which == "bwd":
        assert distill(ops, which, stats=NULL) == inv and distill(ops, which, stats=two) == ali
    if which == "fwd":
        assert distill(ops, which, loss=NULL, stats=NULL) == inv
        assert distill(ops, which, loss=two) == ali
    if which == "both":
        assert distill(ops, which, loss=NULL) == ops.MOE_ERR_NOT_INITIALIZED
