"""fp64 oracle of the projection with bias, activation and residual (plain NumPy and SciPy)."""
import numpy as np
from scipy.special import erfc


def act(z, kind):
    """Value and derivative."""
    if kind == "silu":
        q = np.where(z >= 0, 1 / (1 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1 + np.exp(-np.abs(z))))
        return z * q, q * (1 + z * (1 - q))
    if kind == "gelu":
        phi = 0.5 * erfc(-z / np.sqrt(2.0))
        return z * phi, phi + z * np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
    return z, np.ones_like(z)


def forward(x, w, b, res, kind):
    z = x @ w.T + (0.0 if b is None else b)
    return act(z, kind)[0] + (0.0 if res is None else res), z


def backward(x, w, dy, z, kind):
    dz = dy if kind == "none" else dy * act(z, kind)[1]
    return dz @ w, dz.T @ x, dz.sum(axis=0), dz
