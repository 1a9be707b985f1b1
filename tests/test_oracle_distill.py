"""The distillation loss's definition: its gradient against differences, and
what it reduces to."""
import numpy as np
import pytest

from oracle.distill_oracle import distill


def example(seed, M, V, k, tail):
    g = np.random.default_rng(seed)
    x, t = 2 * g.standard_normal((M, V)), 2 * g.standard_normal((M, k))
    idx = np.stack([g.permutation(V)[:k] for _ in range(M)])
    idx[0, -1] = idx[0, 0]                     # the same token twice
    idx[1, 1:] = -1
    lse = None if not tail else np.logaddexp.reduce(t, axis=1) + g.uniform(0.01, 0.5, M)
    return x, idx, t, lse


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("tau", [1.0, 2.5])
def test_gradient_against_differences(tail, tau):
    x, idx, t, lse = example(1, 4, 9, 4, tail)
    lse = None if lse is None else lse / tau + 3.0
    dloss = np.array([1.0, -0.5, 2.0, 0.25])
    _, dx = distill(x, idx, t, lse, tau, dloss)
    h = 1e-5
    for i in range(x.shape[1]):
        up, down = x.copy(), x.copy()
        up[:, i] += h
        down[:, i] -= h
        d = (distill(up, idx, t, lse, tau)[0] - distill(down, idx, t, lse, tau)[0]) / (2 * h)
        assert np.allclose(dloss * d, dx[:, i], atol=1e-8, rtol=1e-7)


def test_all_tokens_kept_is_the_divergence_of_the_distributions():
    g = np.random.default_rng(3)
    x, t = g.standard_normal((3, 7)), g.standard_normal((3, 7))
    idx = np.tile(np.arange(7), (3, 1))
    p = np.exp(t) / np.exp(t).sum(1, keepdims=True)
    q = np.exp(x) / np.exp(x).sum(1, keepdims=True)
    for lse in (None, np.log(np.exp(t).sum(1))):
        loss, dx = distill(x, idx, t, lse)
        assert np.allclose(loss, (p * np.log(p / q)).sum(1), atol=1e-12)
        assert np.allclose(dx, q - p, atol=1e-12)


def test_rows_without_a_teacher():
    x, idx, t, _ = example(5, 3, 8, 3, False)
    idx[2] = -1
    t[1, 0] = -np.inf                          # its only token
    loss, dx = distill(x, idx, t)
    assert loss[0] > 0 and np.all(loss[1:] == 0) and np.all(dx[1:] == 0)
