"""Tokens that the teacher names several times: loss and gradient are those of
the token named once with the sum of its probabilities, by the fp64 definition of
that.  Tolerances as in test_gpu_distill.py: WORK of the magnitudes that are added (a
token's P log P and its parts' p log p among them: each at most 1 / e a token)."""
import numpy as np
import pytest
import torch

from helpers import gpu_ops
from oracle.distill_oracle import distill

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
WORK = 64 * 2.0 ** -22


@pytest.fixture(scope="module")
def ops():
    return gpu_ops()


def merged(idx, t, tau):
    """every token once, with the log of its summed exponentials"""
    one, s = np.full_like(idx, -1), np.full(t.shape, -1.0)
    for r in range(idx.shape[0]):
        for j, i in enumerate(np.unique(idx[r][idx[r] >= 0])):
            one[r, j], s[r, j] = i, tau * np.logaddexp.reduce(t[r, idx[r] == i] / tau)
    return one, s


# a warp to a row, three warps, parts of a cluster, one wide CTA to a row
@pytest.mark.parametrize("m,v,k", [(650, 1271, 16), (12, 700, 40), (700, 4099, 12), (5, 40001, 64), (3, 129280, 200), (400, 9001, 8)])
@pytest.mark.parametrize("xt", [BF, F])
@pytest.mark.parametrize("tail", [False, True])
def test_as_the_token_named_once(ops, m, v, k, xt, tail):
    tau = 1.0 if m % 2 else 2.0
    g = torch.Generator(device="cuda").manual_seed(k)
    x = (2 * torch.randn((m, v), generator=g, device="cuda")).to(xt)
    idx = torch.randint(v, (m, k), generator=g, device="cuda")
    idx[0] = v - 1                                        # one token throughout
    idx[1, 1::2] = idx[1, :1]                             # half of them
    idx[2:] = torch.where(torch.rand((m - 2, k), generator=g, device="cuda") < 0.5, idx[2:, :1].roll(1, 1), idx[2:])
    idx[2:, k // 2:] = idx[2:, :k - k // 2]               # all of them twice
    idx[-1, -1] = -1
    t = 2 * torch.randn((m, k), generator=g, device="cuda")
    dloss = torch.randn((m,), generator=g, device="cuda")
    idx = idx.to(torch.int32)
    there = torch.where(idx >= 0, t / tau, -torch.inf)
    lse = torch.logsumexp(there, 1) + 0.3 if tail else None
    X, I, T = x.double().cpu().numpy(), idx.cpu().numpy(), t.double().cpu().numpy()
    L = None if lse is None else lse.double().cpu().numpy()
    D = dloss.double().cpu().numpy()
    one, s = merged(I, T, tau)
    loss_w, dx_w = distill(X, one, s, L, tau, D)
    z = X / tau
    top = z.max(1, keepdims=True)
    logq = z - (top + np.log(np.exp(z - top).sum(1, keepdims=True)))
    p = np.exp(there.double().cpu().numpy() - (np.logaddexp.reduce(there.double().cpu().numpy(), axis=1) if L is None else L)[:, None])
    at = np.clip(I, 0, None)
    rows = np.arange(m)[:, None]
    size = tau * tau * ((p * (np.abs(T / tau) + np.abs(z[rows, at]) + np.abs(logq[rows, at]) + 8)).sum(1) + 8 + 2 / np.e * k)
    pull = np.exp(logq) * (2 if L is None else 2 + 1 / 0.5)        # the others have half of q at least
    np.add.at(pull, (rows, at), p)
    pull *= tau * np.abs(D)[:, None] * (1 + np.minimum(np.abs(z - top), 200) / 16)
    tol = np.abs(dx_w) * (2.0 ** -8 if xt == BF else 2.0 ** -24) + WORK * pull + 2.0 ** -120

    def close(a, ref, tol, what):
        off = np.abs(a.double().cpu().numpy() - ref) - tol
        assert np.all(off <= 0), (what, float(off.max()), np.argwhere(off > 0)[:3].tolist())

    loss, stats = ops.distill_loss_fwd(x, idx, t, lse, tau)
    close(loss, loss_w, WORK * size, "loss")
    close(ops.distill_loss_bwd(dloss, x, idx, t, stats, lse, tau), dx_w, tol, "dlogits")
    loss2, d = ops.distill_loss(dloss, x, idx, t, lse, tau)
    close(loss2, loss_w, WORK * size, "loss with gradient")
    close(d, dx_w, tol, "dlogits with loss")
    again, _ = ops.distill_loss(dloss, x, idx, t, lse, tau)
    assert torch.equal(loss2, again)


@pytest.mark.parametrize("m", [1, 700])
def test_a_student_that_equals_the_teacher(ops, m):
    x = torch.log(torch.tensor([[0.5, 0.5]], device="cuda")).repeat(m, 1)
    idx = torch.tensor([[0, 0, 1]], dtype=torch.int32, device="cuda").repeat(m, 1)
    t = torch.log(torch.tensor([[0.25, 0.25, 0.5]], device="cuda")).repeat(m, 1)
    loss, _ = ops.distill_loss_fwd(x, idx, t)
    loss2, d = ops.distill_loss(torch.ones(m, device="cuda"), x, idx, t)
    for a in (loss, loss2, d):
        assert float(a.abs().max()) <= 16 * 2.0 ** -22
