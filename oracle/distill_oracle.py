"""Plain fp64 numpy definition of the distillation loss (test infrastructure
only): the cross entropy of a teacher's kept tokens and of the rest."""
from __future__ import annotations

import numpy as np


def distill(x, idx, t, teacher_lse=None, tau=1.0, dloss=None):
    """(loss [M], dx [M, V]) of logits x, kept tokens idx (negative: none) with
    teacher logits t; dx is the gradient for dloss [M] (ones by default)."""
    x, t = np.asarray(x, np.float64), np.asarray(t, np.float64)
    M, V = x.shape
    loss, dx = np.zeros(M), np.zeros((M, V))
    for r in range(M):
        kept = [j for j in range(idx.shape[1]) if 0 <= idx[r, j] < V]
        if not kept or (teacher_lse is None and np.all(t[r, kept] == -np.inf)):
            continue
        at = np.asarray([idx[r, j] for j in kept])
        zt, z = t[r, kept] / tau, x[r] / tau
        p = np.exp(zt - (np.logaddexp.reduce(zt) if teacher_lse is None else float(teacher_lse[r])))
        logq = z - np.logaddexp.reduce(z)
        target = np.zeros(V)
        np.add.at(target, at, p)
        for i in np.unique(at):              # a token that occurs several times has the sum of its probabilities
            if target[i] > 0:
                loss[r] += target[i] * (np.log(target[i]) - logq[i])
        if teacher_lse is not None:
            others = np.exp(logq)
            others[at] = 0.0
            q_rest, rest = others.sum(), max(1.0 - p.sum(), 0.0)
            if rest > 0 and q_rest > 0:
                loss[r] += rest * (np.log(rest) - np.log(q_rest))
                target += rest * others / q_rest
        loss[r] *= tau * tau
        dx[r] = tau * (np.exp(logq) * target.sum() - target)
    if dloss is not None:
        dx *= np.asarray(dloss, np.float64)[:, None]
        dx[np.asarray(dloss) == 0] = 0.0
    return loss, dx
