"""Matrices of one row, contiguous, of a width that is no multiple of 8: their
stride means nothing and is no reason to refuse them."""
import ctypes

import numpy as np
import pytest
import torch

from helpers import build_lib, gpu_ops

P = ctypes.c_void_p(4096)


@pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers are fake, and the calls are not refused")
def test_the_stride_of_one_row_is_free():
    build_lib()
    from grouped_gemm_top_gb300 import ops
    lib, free, odd = ops.lib, ops.MOE_ERR_NOT_INITIALIZED, ops.MOE_ERR_ALIGNMENT      # (no device here)
    for m, want in ((1, free), (2, odd)):
        assert lib.linear_fwd(P, 65, P, 48, None, 3, P, 41, m, 41, 65, P, 41, P, 41, None, None) == want
        assert lib.linear_bwd(P, 41, P, 65, P, 48, P, 41, 3, m, 41, 65, P, 65, P, 0, 48, P, P, 1 << 20, None, None) == want
        assert lib.gated_ffn_fwd(P, 65, P, 48, 3, m, 24, 65, P, 25, P, 49, None, None) == want
        assert lib.gated_ffn_bwd(P, 25, P, 49, P, 65, P, 48, 3, m, 24, 65, P, 49, P, 65, P, 0, 48, None, None) == want
    # W and its gradient of one row
    assert lib.linear_fwd(P, 8, P, 41, None, 0, None, 0, 5, 41, 1, P, 48, None, 0, None, None) == free
    assert lib.linear_bwd(P, 48, P, 8, P, 41, None, 0, 0, 5, 41, 1, P, 8, P, 1, 41, None, None, 0, None, None) == free
    # a stride shorter than the row is still wrong
    assert lib.linear_fwd(P, 64, P, 48, None, 0, None, 0, 1, 41, 65, P, 41, None, 0, None, None) == ops.MOE_ERR_INVALID_ARG


def t64(t):
    return t.double().cpu().numpy()


@pytest.mark.gpu
@pytest.mark.parametrize("n,k", [(41, 65), (1, 1), (257, 1001), (5003, 99)])
def test_linear_of_one_contiguous_row(n, k):
    """(Tolerances as in test_gpu_dense.py.)"""
    ops = gpu_ops()
    from oracle import dense_oracle as D
    g = torch.Generator(device="cuda").manual_seed(n)

    def row(c):      # one row in the middle of memory that must not change
        buf = torch.randn((16 + c + 16,), generator=g, device="cuda").bfloat16()
        return buf, buf[16:16 + c].view(1, c)

    def same_around(buf, was, c):
        return torch.equal(buf[:16], was[:16]) and torch.equal(buf[16 + c:], was[16 + c:])

    (_, x), (_, r), (yb, y), (zb, z), (_, dy), (dxb, dx) = row(k), row(n), row(n), row(n), row(n), row(k)
    w = torch.randn((k, (n + 7) // 8 * 8), generator=g, device="cuda").mul_(0.1).bfloat16()[:, :n]
    was = yb.clone(), zb.clone(), dxb.clone()
    ops.linear_fwd(x, w, None, "silu", r, y=y, z=z)
    wy, wz = D.linear(t64(x), t64(w), None, "silu", t64(r))
    e = (k / 16 + 8) * 2.0 ** -23 * (np.abs(t64(x)) @ np.abs(t64(w)))
    assert np.all(np.abs(t64(z) - wz) <= e + np.abs(wz) * 2.0 ** -8)
    assert np.all(np.abs(t64(y) - wy) <= 1.2 * e + np.abs(wz) * 2.0 ** -18 + np.abs(t64(r)) * 2.0 ** -22 +
                  np.abs(wy) * (2.0 ** -8 + 2.0 ** -22))
    dw = ops.linear_bwd(dy, x, w, z, "silu", dx=dx, want_dbias=True)[1]
    wdx, wdw, _, dz = D.linear_bwd(t64(dy), t64(x), t64(w), t64(z), "silu")
    rnd = 2.0 ** -8 * np.abs(dz) + np.abs(t64(dy)) * 2.0 ** -18
    a = (n / 16 + 8) * 2.0 ** -23
    assert np.all(np.abs(t64(dx) - wdx) <= np.abs(wdx) * 2.0 ** -8 + (rnd + a * np.abs(dz)) @ np.abs(t64(w)).T)
    assert np.all(np.abs(t64(dw) - wdw) <= np.abs(wdw) * 2.0 ** -8 + np.abs(t64(x)).T @ (rnd + 9 * 2.0 ** -23 * np.abs(dz)))
    assert same_around(yb, was[0], n) and same_around(zb, was[1], n) and same_around(dxb, was[2], k)


@pytest.mark.gpu
@pytest.mark.parametrize("m", [5, 300])
def test_a_weight_of_one_contiguous_row(m):
    ops = gpu_ops()
    g, n = torch.Generator(device="cuda").manual_seed(m), 43
    x = torch.randn((m, 8), generator=g, device="cuda").bfloat16()[:, :1]
    w = torch.randn((1, n), generator=g, device="cuda").bfloat16()
    dy = torch.randn((m, 48), generator=g, device="cuda").bfloat16()[:, :n]
    dw = torch.empty((1, n), device="cuda")
    want = t64(x) @ t64(w)
    assert np.all(np.abs(t64(ops.linear_fwd(x, w)) - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -22))
    ops.linear_bwd(dy, x, w, dw=dw)
    size = np.abs(t64(x)).T @ np.abs(t64(dy))
    assert np.all(np.abs(t64(dw) - t64(x).T @ t64(dy)) <= (m / 16 + 8) * 2.0 ** -23 * size)


@pytest.mark.gpu
def test_gated_forward_and_backward_of_one_contiguous_row():
    """x of odd width alone has to be taken (h and a are multiples of 8 wide)."""
    ops = gpu_ops()
    from oracle import dense_oracle as D
    g, f, d = torch.Generator(device="cuda").manual_seed(1), 264, 129
    x = torch.randn((1, d), generator=g, device="cuda").bfloat16()
    w = torch.randn((d, 2 * f), generator=g, device="cuda").mul_(0.1).bfloat16()
    dh = torch.randn((1, f), generator=g, device="cuda").bfloat16()
    h, a = ops.gated_ffn_fwd(x, w, want_a=True)
    wh, wa = D.gated_ffn(t64(x), t64(w))
    assert np.all(np.abs(t64(a) - wa) <= np.abs(wa) * 2.0 ** -8 + (d / 16 + 8) * 2.0 ** -23 * (np.abs(t64(x)) @ np.abs(t64(w))))
    assert np.linalg.norm(t64(h) - wh) <= 2.0 ** -8 * np.linalg.norm(wh)
    dx = torch.empty((1, d), dtype=torch.bfloat16, device="cuda")
    _, dw = ops.gated_ffn_bwd(dh, a, x, w, dx=dx)
    wdx, wdw, _ = D.gated_ffn_bwd(t64(dh), t64(a), t64(x), t64(w))
    assert np.linalg.norm(t64(dx) - wdx) <= 2.0 ** -8 * np.linalg.norm(wdx)
    assert np.linalg.norm(t64(dw) - wdw) <= 2.0 ** -7 * np.linalg.norm(wdw)      # da's rounding and its own
