"""The distillation loss with the teacher's whole log-sum-exp where the student
is sure of the kept tokens: the others lie up to 600 temperatures below them, or are
masked.  Against the fp64 definition.

Tolerances as in test_gpu_distill.py: a probability whose exponent is `a` is off by
(2 + a + 40) 2^-22 of its value, at most (1 + a / 16) WORK; rest, as 1 - mass, by
WORK of the mass; sums by WORK of the magnitudes that are added.  The backward call
takes the kept tokens relative to a log-sum-exp that is rounded once, 2^-24 of its
exponent.  A bf16 result is off by half a step besides."""
import numpy as np
import pytest
import torch

from helpers import gpu_ops
from oracle.distill_oracle import distill

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
WORK = 64 * 2.0 ** -22

# a warp to a row (two types' longest), three warps, a cluster or one wide CTA to a row
SIZES = [(650, 1271), (12, 2551), (700, 4099), (400, 9001), (7, 32001), (9, 50257)]


@pytest.fixture(scope="module")
def ops():
    return gpu_ops()


def example(m, v, xt, gap, tau, k=8):
    """the kept tokens `gap` above the others, but for rows 1 (ordinary), 2 (the others above the kept), 3 (a third of
    the others -inf), 4 (all), 5 (all of the type's lowest value), 6 (no teacher)"""
    g = torch.Generator(device="cuda").manual_seed(v)
    x = torch.randn((m, v), generator=g, device="cuda") * min(tau, 1.0)
    idx = torch.stack([torch.randperm(v, generator=g, device="cuda")[:k] for _ in range(m)])
    step = torch.full((m, 1), float(gap), device="cuda")
    step[1], step[2] = 0.0, -gap
    kept = torch.zeros((m, v), dtype=torch.bool, device="cuda").scatter_(1, idx, True)
    x = torch.where(kept, x + step / 2, x - step / 2)
    third = torch.arange(v, device="cuda") % 3 == 0
    x[3] = torch.where(third & ~kept[3], -torch.inf, x[3])
    x[4] = torch.where(kept[4], x[4], -torch.inf)
    x[5] = torch.where(kept[5], x[5], torch.finfo(xt).min)
    idx[6] = -1
    t = torch.randn((m, k), generator=g, device="cuda") * 2
    lse = torch.logsumexp(t / tau, 1) + 0.3 * torch.rand((m,), generator=g, device="cuda") + 0.01
    dloss = torch.randn((m,), generator=g, device="cuda")
    return x.to(xt), idx.to(torch.int32), t, lse, dloss


def np64(t):
    return t.double().cpu().numpy()


def want(x, idx, t, lse, tau, dloss):
    """loss, gradient and the magnitudes that their errors are relative to"""
    X, I, T, L, D = np64(x), idx.cpu().numpy(), np64(t), np64(lse), np64(dloss)
    loss, dx = distill(X, I, T, L, tau, D)
    z = np.maximum(X, -1e30) / tau
    top = z.max(1, keepdims=True)
    logq = z - (top + np.log(np.exp(z - top).sum(1, keepdims=True)))
    size, pull = np.zeros_like(loss), np.zeros_like(dx)
    for r in range(X.shape[0]):
        kept = I[r][I[r] >= 0]
        if kept.size == 0:
            continue
        p = np.exp(T[r] / tau - L[r])
        others = np.ones(X.shape[1], bool)
        others[kept] = False
        zo = z[r, others]
        share = np.exp(zo - zo.max())
        log_rest = zo.max() + np.log(share.sum()) - (z[r, kept[0]] - logq[r, kept[0]])
        log_rest = 0.0 if log_rest < -745 else log_rest
        size[r] = tau * tau * (np.sum(p * (np.abs(T[r] / tau) + np.abs(z[r, kept]) + np.abs(logq[r, kept]) + 8)) + 8 + abs(log_rest))
        pull[r] = np.exp(logq[r]) * (1 + np.minimum(np.abs(z[r] - top[r]), 100) / 16)
        pull[r, kept] += p + np.exp(logq[r, kept]) * abs(top[r, 0]) / 64
        if log_rest != 0:
            pull[r, others] += share / share.sum() * (1 + np.minimum(zo.max() - zo, 100) / 16)
        pull[r] *= tau * abs(D[r])
    return loss, dx, WORK * size, WORK * pull


def close(got, ref, tol, what):
    g = np64(got)
    assert np.all(np.isfinite(g)), (what, np.argwhere(~np.isfinite(g))[:3].tolist())
    off = np.abs(g - ref) - tol - 2.0 ** -120
    assert np.all(off <= 0), (what, float(off.max()), np.argwhere(off > 0)[:3].tolist())


def check(ops, x, idx, t, lse, dloss, tau):
    loss_w, dx_w, loss_tol, pull = want(x, idx, t, lse, tau, dloss)
    tol = np.abs(dx_w) * (2.0 ** -8 if x.dtype == BF else 2.0 ** -24) + pull
    loss, stats = ops.distill_loss_fwd(x, idx, t, lse, tau)
    close(loss, loss_w, loss_tol, "loss")
    close(ops.distill_loss_bwd(dloss, x, idx, t, stats, lse, tau), dx_w, tol, "dlogits")
    loss2, d = ops.distill_loss(dloss, x, idx, t, lse, tau)
    close(loss2, loss_w, loss_tol, "loss with gradient")
    close(d, dx_w, tol, "dlogits with loss")
    return loss2, d


@pytest.mark.parametrize("m,v", SIZES)
@pytest.mark.parametrize("xt", [BF, F])
@pytest.mark.parametrize("gap,tau", [(36, 1.0), (44, 1.0), (60, 1.0), (90, 1.0), (150, 1.0), (24, 0.25), (150, 0.25), (300, 2.0)])
def test_others_far_below(ops, m, v, xt, gap, tau):
    args = example(m, v, xt, gap, tau)
    check(ops, *args, tau)


@pytest.mark.parametrize("xt", [BF, F])
@pytest.mark.parametrize("gap", [80, 87, 90, 150])
def test_large_weights(ops, xt, gap):
    """a loss scale: no overflow on the way to the gradient"""
    for m, v in ((650, 1271), (7, 32001)):
        x, idx, t, lse, dloss = example(m, v, xt, gap, 1.0)
        check(ops, x, idx, t, lse, dloss * 65536.0 ** 2, 1.0)


@pytest.mark.parametrize("xt", [BF, F])
def test_in_place_and_again(ops, xt):
    for m, v in ((650, 1271), (700, 4099), (7, 32001)):
        x, idx, t, lse, dloss = example(m, v, xt, 120, 1.0)
        loss, d = ops.distill_loss(dloss, x, idx, t, lse)
        _, stats = ops.distill_loss_fwd(x, idx, t, lse)
        e = ops.distill_loss_bwd(dloss, x, idx, t, stats, lse)
        y, z = x.clone(), x.clone()
        again, _ = ops.distill_loss(dloss, y, idx, t, lse, dlogits=y)
        ops.distill_loss_bwd(dloss, z, idx, t, stats, lse, dlogits=z)
        assert torch.equal(loss, again) and torch.equal(d, y) and torch.equal(e, z)


def test_gradient_against_differences(ops):
    """of the rows' losses in 64 bits by the definition, for kept tokens and others"""
    x, idx, t, lse, dloss = example(7, 300, F, 100, 1.0)
    _, d = ops.distill_loss(dloss, x, idx, t, lse)
    X, I, T, L, h = np64(x), idx.cpu().numpy(), np64(t), np64(lse), 1e-4
    scale = np.abs(np64(d)).max(1)
    for r in (0, 1, 2, 3):
        for i in (int(I[r, 0]), int(I[r, 5]), 7, 200, 299):
            if not np.isfinite(X[r, i]):
                continue
            up, down = X.copy(), X.copy()
            up[r, i] += h
            down[r, i] -= h
            diff = (distill(up, I, T, L)[0][r] - distill(down, I, T, L)[0][r]) / (2 * h) * float(dloss[r])
            assert abs(diff - float(d[r, i])) <= 1e-5 * scale[r], (r, i)
