"""The square root of the second moment over every magnitude fp32 holds."""
import numpy as np
import pytest
import torch

from helpers import gpu_ops

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ops():
    return gpu_ops()


def values(n, lo, hi, seed):
    """n positive fp32 with exponents spread over [lo, hi], subnormals as they fall."""
    r = np.random.default_rng(seed)
    return np.ldexp(r.uniform(1, 2, n), r.integers(lo, hi + 1, n)).astype(np.float32)


@pytest.mark.parametrize("dense", [True, False])      # the elements beside it alike, or zeros
def test_stored_roots_are_correctly_rounded(ops, dense):
    """With b2 = 0, v is the gradient's square, and a block's scale is its
    largest root over 448: the root's own bits can be told."""
    g = np.concatenate([values(60000, -74, 63, 1), np.float32([1e-22, 2.0 ** -74, 2.0 ** -50, 1.5 * 2.0 ** -50, 2.0 ** 63])])
    blocks = len(g)
    grad = torch.zeros((blocks, 256), device="cuda")
    col = torch.from_numpy(g).cuda()
    if dense:
        grad[:] = col[:, None]
    else:
        grad[torch.arange(blocks), torch.arange(blocks) * 37 % 256] = col
    n = blocks * 256
    p, z = torch.zeros((n,), dtype=BF, device="cuda"), lambda t, k: torch.zeros((k,), dtype=t, device="cuda")
    m, v, ms, vs = z(torch.uint8, n), z(torch.uint8, n), z(F, blocks), z(F, blocks)
    plan = ops.adamw_plan([p], [grad.view(-1)], [m], [v], [ms], [vs])
    ops.adamw_step(plan, 0.0, (0.9, 0.0), 1e-8, step=1)
    with np.errstate(under="ignore"):
        want = np.sqrt(g * g) * np.float32(1 / 448)
    got = vs.cpu().numpy()
    assert got.dtype == want.dtype == np.float32
    bad = np.flatnonzero(got != want)
    assert len(bad) == 0, (len(bad), g[bad[:4]], got[bad[:4]], want[bad[:4]])
    assert not v.view(blocks, 256)[:, :][grad == 0].any()


@pytest.mark.parametrize("gt", [F, BF])
def test_update_without_eps(ops, gt):
    """p = -m / sqrt(v) with m = 1: the root's half step, 2^-22 of the approximate
    reciprocal (its bound on [1, 2], 2^-23, over results from 1/2), the product's half step."""
    v0 = np.concatenate([values(200000, -149, 126, 2), np.float32(2.0) ** np.arange(-148, 127, dtype=np.float32),
                         np.float32([1e-39, 1e-40, 1.4e-45 * 2, 1.1754944e-38, 2.0 ** -100, 2.0 ** -99])])
    n = len(v0)
    p, g = torch.zeros((n,), device="cuda"), torch.zeros((n,), dtype=gt, device="cuda")
    m, v = torch.full((n,), 2.0, device="cuda"), torch.from_numpy(v0).cuda()
    ops.adamw_step(ops.adamw_plan([p], [g], [m], [v]), 1.0, (0.5, 0.5), 0.0, step=1000)
    with np.errstate(under="ignore"):
        v1 = np.float32(0.5) * v0
    assert np.array_equal(v.cpu().numpy(), v1)
    some = v1 > 0
    want = -1 / np.sqrt(v1[some].astype(np.float64))
    off = np.abs(p.double().cpu().numpy()[some] / want - 1)
    assert off.max() <= (2.0 ** -24 + 2.0 ** -22 + 2.0 ** -24) * 1.001, (off.max(), v1[some][off.argmax()])
