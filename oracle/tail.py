"""The tail of an update step: fp64 oracle.

TEST INFRASTRUCTURE ONLY.  Nothing on the product path imports this module; only ``tests/``
do.  It shares no code with the library.

RMS norm with the residual's addition (forward, backward, 8-bit blocks), the gradients'
global norm and clipping, and log-probabilities from hidden rows and the vocabulary weight
(the logits are formed here and given to the compact-to-semantic oracle)."""
from __future__ import annotations

import numpy as np

from . import logprob


def rmsnorm_fwd(x, residual, weight, eps):
    """(y, h, rstd) in fp64."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + np.asarray(residual, np.float64)
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    return h * rstd[:, None] * np.asarray(weight, np.float64), h, rstd


def rmsnorm_bwd(dy, h, weight, rstd, dh=None):
    """(dx, dweight) for y = h rstd weight with rstd a function of h."""
    dy, h, w = (np.asarray(a, np.float64) for a in (dy, h, weight))
    r = np.asarray(rstd, np.float64)[:, None]
    n = h * r
    t = dy * w
    dx = r * (t - n * (t * n).mean(axis=1, keepdims=True))
    if dh is not None:
        dx = dx + np.asarray(dh, np.float64)
    return dx, (dy * n).sum(axis=0)


def mx_scales(y, block=32):
    """The smallest power of two per block of a row that keeps the block within 448; 2^-127
    is the smallest there is."""
    y = np.asarray(y, np.float64)
    amax = np.abs(y.reshape(y.shape[0], -1, block)).max(axis=2)
    with np.errstate(divide="ignore"):
        e = np.ceil(np.log2(amax / 448.0))
    return np.exp2(np.clip(e, -127, 127))


def grad_clip(grads, max_norm):
    """(norm, clipped gradients)."""
    norm = np.sqrt(sum(float((np.asarray(g, np.float64) ** 2).sum()) for g in grads))
    coef = max_norm / norm if np.isfinite(norm) and norm > max_norm else 1.0
    return norm, [np.asarray(g, np.float64) * coef for g in grads]


def _positions(sem_row, target, V):
    """Positions that have a label."""
    target = np.asarray(target)
    keep = (target >= 0) & (target < V)
    return keep, np.asarray(sem_row)[keep], target[keep]


def linear_logprob_fwd(x, weight, sem_row, target, scale=1.0):
    """(logp [S], lse [C]); logp is 0 where the target lies outside the vocabulary."""
    z = scale * (np.asarray(x, np.float64) @ np.asarray(weight, np.float64).T)
    keep, rows, labels = _positions(sem_row, target, z.shape[1])
    lam, lse = logprob.logprob_fwd(z, rows, labels)
    logp = np.zeros(len(keep))
    logp[keep] = lam
    return logp, lse


def linear_logprob_bwd(x, weight, sem_row, target, g, scale=1.0):
    """(dx, dweight) of sum_s g_s logp[s]."""
    x, w = np.asarray(x, np.float64), np.asarray(weight, np.float64)
    keep, rows, labels = _positions(sem_row, target, w.shape[0])
    dz = logprob.logprob_bwd(scale * (x @ w.T), rows, labels, np.asarray(g, np.float64)[keep])
    return scale * (dz @ w), scale * (dz.T @ x)
