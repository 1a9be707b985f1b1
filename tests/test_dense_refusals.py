"""Host-side checks of the dense operators' C entry points: every call here
is refused (or has nothing to do) before any device work, the pointers are
fake."""
import ctypes

import pytest

from helpers import build_lib


@pytest.fixture(scope="module")
def ops():
    build_lib()
    from grouped_gemm_top_gb300 import ops
    return ops


P, ODD, NULL = ctypes.c_void_p(4096), ctypes.c_void_p(4097), None


def norm_fwd(ops, **k):
    a = dict(x=P, xt=0, ldx=256, res=P, rt=0, ldres=256, w=P, wt=0, eps=1e-6, M=4, N=256, r=P, ldr=256, y=P, yt=0,
             ldy=256, rstd=P, codes=P, scales=P, sf=ops.MOE_SF_ATOMS)
    a.update(k)
    return ops.lib.rmsnorm_residual_fwd(*a.values(), NULL)


def test_norm_forward(ops):
    inv, uns, ali = ops.MOE_ERR_INVALID_ARG, ops.MOE_ERR_UNSUPPORTED, ops.MOE_ERR_ALIGNMENT
    for k in (dict(x=NULL), dict(w=NULL), dict(M=-1), dict(N=0), dict(xt=2), dict(rt=-1), dict(wt=9), dict(yt=5),
              dict(ldx=255), dict(ldres=0), dict(ldr=255), dict(ldy=255), dict(eps=-1.0), dict(codes=NULL),
              dict(scales=NULL), dict(sf=ops.MOE_SF_TILE224), dict(eps=float("nan"))):
        assert norm_fwd(ops, **k) == inv, k
    assert norm_fwd(ops, r=NULL, y=NULL, rstd=NULL, codes=NULL, scales=NULL) == inv
    wide = dict(ldx=40000, ldres=40000, ldr=40000, ldy=40000)
    assert norm_fwd(ops, N=32769, **wide) == uns
    assert norm_fwd(ops, N=160) == uns
    assert norm_fwd(ops, N=48, sf=ops.MOE_SF_CANONICAL) == uns
    assert norm_fwd(ops, M=1 << 31) == uns
    for k in (dict(x=ODD), dict(res=ODD), dict(w=ODD), dict(r=ODD), dict(y=ODD), dict(rstd=ODD), dict(codes=ODD)):
        assert norm_fwd(ops, **k) == ali, k
    assert norm_fwd(ops, M=0, x=NULL, y=NULL, r=NULL, rstd=NULL, res=NULL) == ops.MOE_OK


def norm_bwd(ops, **k):
    a = dict(dy=P, dyt=0, lddy=256, r=P, rt=0, ldr=256, w=P, wt=0, rstd=P, dres=P, lddres=256, M=4, N=256, dx=P,
             lddx=256, dw=P, ws=P, wsb=1 << 30)
    a.update(k)
    return ops.lib.rmsnorm_residual_bwd(*a.values(), NULL)


def test_norm_backward(ops):
    inv = ops.MOE_ERR_INVALID_ARG
    for k in (dict(dy=NULL), dict(r=NULL), dict(w=NULL), dict(rstd=NULL), dict(dx=NULL), dict(M=-1), dict(N=0),
              dict(dyt=2), dict(rt=2), dict(wt=2), dict(lddy=255), dict(ldr=255), dict(lddx=255), dict(lddres=255)):
        assert norm_bwd(ops, **k) == inv, k
    assert norm_bwd(ops, ws=NULL) == ops.MOE_ERR_WORKSPACE
    assert norm_bwd(ops, wsb=4 * 256 * 4 - 1) == ops.MOE_ERR_WORKSPACE
    for k in (dict(dy=ODD), dict(r=ODD), dict(w=ODD), dict(dres=ODD), dict(dx=ODD), dict(dw=ODD), dict(ws=ODD)):
        assert norm_bwd(ops, **k) == ops.MOE_ERR_ALIGNMENT, k
    assert ops.rmsnorm_bwd_workspace_size(4, 256) == 4 * 256 * 4
    assert ops.rmsnorm_bwd_workspace_size(5, 256) == 8 * 256 * 4          # short rows: four to a CTA
    assert ops.rmsnorm_bwd_workspace_size(1 << 20, 4096) == 608 * 4096 * 4
    assert ops.rmsnorm_bwd_workspace_size(0, 4096) == 0
    assert ops.rmsnorm_bwd_workspace_size(-1, 4096) == -1 and ops.rmsnorm_bwd_workspace_size(4, 1 << 20) == -1


def encode(ops, n=1, p=4096, g=4096, m=4096, v=4096, ms=4096, vs=4096, copy=None, numel=1000, rng=0, pt=1, gt=0,
           bits=8):
    arr = (ops.AdamWTensor * max(n, 1))()
    for i in range(max(n, 1)):
        arr[i] = ops.AdamWTensor(p, g, m, v, ms, vs, copy, numel, rng, 0.1)
    buf = (ctypes.c_int64 * 64)()
    tiles = ctypes.c_int64(-1)
    st = ops.lib.adamw_plan_encode(ctypes.cast(arr, ctypes.c_void_p), n, pt, gt, bits, ctypes.cast(buf, ctypes.c_void_p),
                                   ctypes.byref(tiles))
    return st, tiles.value


def test_adamw(ops):
    inv, ali = ops.MOE_ERR_INVALID_ARG, ops.MOE_ERR_ALIGNMENT
    assert encode(ops) == (ops.MOE_OK, 1)
    assert encode(ops, n=3, numel=2049) == (ops.MOE_OK, 6)
    assert encode(ops, numel=0, p=None, g=None) == (ops.MOE_OK, 0)
    for k in (dict(n=0), dict(p=None), dict(g=None), dict(m=None), dict(v=None), dict(ms=None), dict(vs=None),
              dict(numel=-1), dict(rng=8), dict(rng=-256), dict(pt=2), dict(gt=7), dict(bits=16)):
        assert encode(ops, **k)[0] == inv, k
    for k in (dict(p=4098), dict(g=4097), dict(ms=4098), dict(vs=4097), dict(copy=4097), dict(bits=32, m=4098)):
        assert encode(ops, **k)[0] == ali, k
    assert encode(ops, bits=32, ms=None, vs=None) == (ops.MOE_OK, 1)
    assert ops.lib.adamw_plan_bytes(1) == 16 + 80 + 16
    assert ops.lib.adamw_plan_bytes(0) == ctypes.c_size_t(-1).value

    def step(plan=P, tensors=1, tiles=1, pt=1, gt=0, bits=8, opts=True, **k):
        o = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, step=1, step_dev=None, lr_dev=None, grad_scale=None, seed=0)
        o.update(k)
        return ops.lib.adamw_step(plan, tensors, tiles, pt, gt, bits, ctypes.byref(ops.AdamWOpts(*o.values())) if opts else None,
                                  NULL)
    for k in (dict(plan=NULL), dict(tensors=0), dict(tiles=-1), dict(pt=3), dict(gt=-1), dict(bits=4), dict(opts=False),
              dict(beta1=1.0), dict(beta2=-0.1), dict(eps=-1.0), dict(step=0)):
        assert step(**k) == inv, k
    for k in (dict(plan=ctypes.c_void_p(4104)), dict(step_dev=4097), dict(lr_dev=4098), dict(grad_scale=4097)):
        assert step(**k) == ali, k


def lin_fwd(ops, **k):
    a = dict(x=P, ldx=64, w=P, ldw=48, bias=P, act=1, res=P, ldres=48, M=16, N=48, K=64, y=P, ldy=48, z=P, ldz=48)
    a.update(k)
    return ops.lib.linear_fwd(*a.values(), NULL, NULL)


def lin_bwd(ops, **k):
    a = dict(dy=P, lddy=48, x=P, ldx=64, w=P, ldw=48, z=P, ldz=48, act=3, M=16, N=48, K=64, dx=P, lddx=64, dw=P, dwt=0,
             lddw=48, db=P, ws=P, wsb=1 << 30)
    a.update(k)
    return ops.lib.linear_bwd(*a.values(), NULL, NULL)


def ffn_fwd(ops, **k):
    a = dict(x=P, ldx=64, w=P, ldw=48, act=3, M=16, f=24, d=64, h=P, ldh=24, a=P, lda=48)
    a.update(k)
    return ops.lib.gated_ffn_fwd(*a.values(), NULL, NULL)


def ffn_bwd(ops, **k):
    a = dict(dh=P, lddh=24, a=P, lda=48, x=P, ldx=64, w=P, ldw=48, act=3, M=16, f=24, d=64, da=P, ldda=48, dx=P, lddx=64,
             dw=P, dwt=1, lddw=48)
    a.update(k)
    return ops.lib.gated_ffn_bwd(*a.values(), NULL, NULL)


@pytest.mark.parametrize("call,invalid,unaligned,unsupported", [
    (lin_fwd, [dict(x=NULL), dict(w=NULL), dict(y=NULL), dict(M=-1), dict(N=0), dict(K=0), dict(act=4), dict(act=-1),
               dict(ldx=63), dict(ldw=47), dict(ldy=47), dict(ldz=47), dict(ldres=47)],
     [dict(x=ODD), dict(w=ODD), dict(y=ODD), dict(z=ODD), dict(res=ODD), dict(bias=ODD), dict(ldx=65), dict(ldw=49),
      dict(ldy=49), dict(ldz=49), dict(ldres=49), dict(N=41, ldy=41)], [dict(M=1 << 31)]),
    (lin_bwd, [dict(dy=NULL), dict(x=NULL), dict(w=NULL), dict(z=NULL), dict(M=-1), dict(act=4), dict(dwt=2), dict(lddy=47),
               dict(ldx=63), dict(ldw=47), dict(ldz=47), dict(lddx=63), dict(lddw=47), dict(dx=NULL, dw=NULL, db=NULL)],
     [dict(dy=ODD), dict(x=ODD), dict(w=ODD), dict(z=ODD), dict(dx=ODD), dict(dw=ODD), dict(db=ODD), dict(ws=ODD),
      dict(lddy=49), dict(lddx=65)], [dict(M=1 << 31)]),
    (ffn_fwd, [dict(x=NULL), dict(w=NULL), dict(h=NULL), dict(M=-1), dict(f=0), dict(d=0), dict(act=9), dict(ldx=63),
               dict(ldw=47), dict(ldh=23), dict(lda=47)],
     [dict(x=ODD), dict(w=ODD), dict(h=ODD), dict(a=ODD), dict(ldh=25), dict(lda=50)], [dict(f=20), dict(M=1 << 31)]),
    (ffn_bwd, [dict(dh=NULL), dict(a=NULL), dict(x=NULL), dict(w=NULL), dict(da=NULL), dict(M=-1), dict(dwt=-1), dict(lddh=23),
               dict(lda=47), dict(ldda=47), dict(ldx=63), dict(ldw=47), dict(lddx=63), dict(lddw=47)],
     [dict(dh=ODD), dict(a=ODD), dict(da=ODD), dict(x=ODD), dict(w=ODD), dict(dx=ODD), dict(dw=ODD), dict(lddw=49)],
     [dict(f=20), dict(M=1 << 31)]),
])
def test_dense_layers(ops, call, invalid, unaligned, unsupported):
    for k in invalid:
        assert call(ops, **k) == ops.MOE_ERR_INVALID_ARG, k
    for k in unaligned:
        assert call(ops, **k) == ops.MOE_ERR_ALIGNMENT, k
    for k in unsupported:
        assert call(ops, **k) == ops.MOE_ERR_UNSUPPORTED, k


def test_dense_workspace_and_no_rows(ops):
    assert lin_bwd(ops, ws=NULL) == ops.MOE_ERR_WORKSPACE
    assert lin_bwd(ops, wsb=ops.linear_bwd_workspace_size(16, 48) - 1) == ops.MOE_ERR_WORKSPACE
    assert ops.linear_bwd_workspace_size(16, 48) == 16 * 48 * 2 + 48 * 4
    assert ops.linear_bwd_workspace_size(-1, 48) == -1 and ops.linear_bwd_workspace_size(16, 0) == -1
    assert lin_fwd(ops, M=0, x=NULL, y=NULL, z=NULL, res=NULL) == ops.MOE_OK
    assert ffn_fwd(ops, M=0, x=NULL, h=NULL, a=NULL) == ops.MOE_OK
