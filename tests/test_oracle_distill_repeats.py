"""A token that the teacher names several times has the sum of its
probabilities, in the definition's loss as in its gradient."""
import numpy as np
import pytest

from oracle.distill_oracle import distill


def test_a_student_that_equals_the_teacher():
    x = np.log([[0.5, 0.5]])
    loss, dx = distill(x, np.array([[0, 0, 1]]), np.log([[0.25, 0.25, 0.5]]))
    assert np.allclose(loss, 0, atol=1e-15) and np.allclose(dx, 0, atol=1e-15)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("tau", [0.5, 1.0, 3.0])
def test_as_the_token_named_once(tail, tau):
    g = np.random.default_rng(7)
    x, t = 2 * g.standard_normal((2, 12)), 2 * g.standard_normal((2, 5))
    idx = np.array([[3, 9, 3, 1, 3], [5, 5, 5, 5, 5]])
    once = np.array([[3, 9, 1, -1, -1], [5, -1, -1, -1, -1]])
    s = np.zeros((2, 5))
    s[0, 0] = tau * np.logaddexp.reduce(t[0, [0, 2, 4]] / tau)
    s[0, 1:3] = t[0, [1, 3]]
    s[1, 0] = tau * np.logaddexp.reduce(t[1] / tau)
    lse = np.logaddexp.reduce(t / tau, axis=1) + 0.2 if tail else None
    for a, b in zip(distill(x, idx, t, lse, tau), distill(x, once, s, lse, tau)):
        assert np.allclose(a, b, rtol=1e-12, atol=1e-13)
