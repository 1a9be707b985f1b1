"""AdamW over weights and gradients that lie in rows with padding between
them, as a linear layer of odd width has them."""
import numpy as np
import pytest
import torch

from helpers import gpu_ops
from oracle import dense_oracle as D

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ops():
    return gpu_ops()


def f64(t):
    return t.double().cpu().numpy()


def rows(m, n, seed, std, pad, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.randn((m, n + pad), generator=g, device="cuda").mul_(std).to(dtype)
    buf[:, n:] = float("nan")
    return buf[:, :n]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("m,n,pad_p,pad_g,gdtype", [(72, 41, 7, 7, BF), (40, 257, 7, 0, BF), (3, 5001, 0, 7, F),
                                                    (30, 4099, 5, 13, F), (1, 41, 7, 7, BF)])
def test_padded_rows_are_updated_in_place(ops, bits, m, n, pad_p, pad_g, gdtype):
    """As the formula says, from the gradient's present values, in every step;
    the bits of the same tensors without padding; nothing between the rows.
    (32 bits: fp32 chains, 2^-21 of the update and of the value.)"""
    from grouped_gemm_top_gb300.optim import AdamW
    p, g = rows(m, n, 1, 0.02, pad_p), rows(m, n, 2, 1e-3, pad_g, gdtype)
    q, h = [t.clone() for t in p.unbind(0)], [t.clone() for t in g.unbind(0)]      # row by row, each on its own
    a = AdamW([(p, g)], 1e-2, weight_decay=0.1, state_bits=bits, seed=7)
    b = AdamW(list(zip(q, h)), 1e-2, weight_decay=0.1, state_bits=bits, seed=7)
    want, mm, vv = f64(p), np.zeros((m, n)), np.zeros((m, n))
    for t in (1, 2, 3):
        a.step_()
        b.step_()
        want, mm, vv = D.adamw(want, f64(g), mm, vv, t, 1e-2, 0.9, 0.999, 1e-8, 0.1)
        if bits == 32:
            got = f64(a.masters[0]).reshape(m, n)
            assert np.all(np.abs(got - want) <= t * (2.0 ** -21 * np.abs(want) + 1e-2 * 2.0 ** -16))
        assert torch.equal(p, a.masters[0].view(m, n).to(BF))
        assert all(torch.equal(x, y) for x, y in zip(p.unbind(0), q))
        fresh = torch.randn((m, n), generator=torch.Generator(device="cuda").manual_seed(t), device="cuda") * 1e-3
        g.copy_(fresh)
        for x, y in zip(h, g.unbind(0)):
            x.copy_(y)
    for t in (p, g):
        if t._base is not None and not t.is_contiguous():
            assert torch.isnan(t._base[:, n:]).all()


def test_a_layer_of_odd_width_learns(ops):
    """linear_fwd / linear_bwd allocate and demand padded rows at width 41."""
    from grouped_gemm_top_gb300.optim import AdamW
    m, k, n = 192, 64, 41
    x, w, target = rows(m, k, 1, 1.0, 0), rows(k, n, 2, 0.1, 7), rows(m, n, 3, 1.0, 7)
    dy, y = rows(m, n, 4, 1.0, 7), rows(m, n, 6, 1.0, 7)
    dw = ops.linear_bwd(dy, x, w, want_dx=False)[1]
    assert not w.is_contiguous() and not dw.is_contiguous()
    opt = AdamW([(w, dw)], 1e-2)
    losses = []
    for _ in range(30):
        ops.linear_fwd(x, w, y=y)
        e = y.float() - target.float()
        losses.append(float(e.square().mean()))
        dy.copy_(e)
        ops.linear_bwd(dy, x, w, want_dx=False, dw=dw)
        opt.step_()
    assert losses[-1] < 0.9 * losses[0] and all(np.isfinite(losses))
