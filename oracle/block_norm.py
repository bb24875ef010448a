"""fp64 oracle of the norms around a block with its gate and residual (plain NumPy)."""
import numpy as np


def gate(z, act):
    """Value and derivative."""
    if act == "linear":
        return z, np.ones_like(z)
    q = np.where(z >= 0, 1 / (1 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1 + np.exp(-np.abs(z))))
    if act == "sigmoid":
        return q, q * (1 - q)
    return z * q, q * (1 + z * (1 - q))


def forward(y, post, g, act, scale, res, pre, eps):
    """(h, n, rstd_post, rstd_pre); absent inputs and outputs are None."""
    r1 = r2 = n = None
    u = y
    if post is not None:
        r1 = 1 / np.sqrt(np.mean(y * y, axis=1) + eps)
        u = y * r1[:, None] * post
    h = scale * u * (1.0 if g is None else gate(g, act)[0]) + (0.0 if res is None else res)
    if pre is not None:
        r2 = 1 / np.sqrt(np.mean(h * h, axis=1) + eps)
        n = h * r2[:, None] * pre
    return h, n, r1, r2


def backward(y, h, dn, dh, post, g, act, scale, pre, r1, r2):
    """dict of dy, dresidual, dgate, dpost_weight, dpre_weight, and d_block (the gradient of the
    gated block's normed output), from the forward's h and reciprocal roots."""
    out = {}
    d = np.zeros_like(y) if dh is None else dh
    if pre is not None:
        N = h * r2[:, None]
        t = dn * pre
        d = d + r2[:, None] * (t - N * np.mean(t * N, axis=1, keepdims=True))
        out["dpre_weight"] = np.sum(dn * N, axis=0)
    out["dresidual"] = d
    Y = y if post is None else y * r1[:, None]
    u = Y if post is None else Y * post
    value, slope = (np.ones_like(y), None) if g is None else gate(g, act)
    if g is not None:
        out["dgate"] = scale * d * u * slope
    e = scale * d * value
    out["d_block"] = e
    if post is None:
        out["dy"] = e
    else:
        t = e * post
        out["dpost_weight"] = np.sum(e * Y, axis=0)
        out["dy"] = r1[:, None] * (t - Y * np.mean(t * Y, axis=1, keepdims=True))
    return out
