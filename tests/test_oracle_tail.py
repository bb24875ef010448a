"""Pins for the update-tail oracle (oracle/tail.py): finite differences of both backward
passes, the 8-bit scales against a search, and the clipping's definition."""
import numpy as np
import pytest

from oracle import tail


def _differences(f, a, eps=1e-6):
    num = np.zeros_like(a)
    for i in np.ndindex(a.shape):
        a0 = a[i]
        a[i] = a0 + eps; hi = f()
        a[i] = a0 - eps; lo = f()
        a[i] = a0
        num[i] = (hi - lo) / (2 * eps)
    return num


@pytest.mark.parametrize("residual", [False, True])
def test_rmsnorm_backward_finite_differences(residual):
    rng = np.random.default_rng(1)
    C, D, eps = 3, 7, 1e-3
    x, w = rng.standard_normal((C, D)), rng.standard_normal(D)
    r = rng.standard_normal((C, D)) if residual else None
    dy, dh = rng.standard_normal((C, D)), rng.standard_normal((C, D))

    def loss():
        y, h, _ = tail.rmsnorm_fwd(x, r, w, eps)
        return float((y * dy).sum() + (h * dh).sum())

    _, h, rstd = tail.rmsnorm_fwd(x, r, w, eps)
    dx, dw = tail.rmsnorm_bwd(dy, h, w, rstd, dh)
    np.testing.assert_allclose(dx, _differences(loss, x), atol=1e-7)
    if residual:
        np.testing.assert_allclose(dx, _differences(loss, r), atol=1e-7)
    np.testing.assert_allclose(dw, _differences(loss, w), atol=1e-7)


def test_mx_scales_are_the_smallest_that_fit():
    rng = np.random.default_rng(2)
    y = rng.standard_normal((40, 64)) * np.exp(rng.standard_normal((40, 1)) * 20)
    y[0, :32] = 0
    y[1, 0], y[1, 1:32] = 448.0, 0.0                     # exactly the largest value
    y[2, 0], y[2, 1:32] = np.nextafter(448.0, 1e9), 0.0  # just over it
    s = tail.mx_scales(y)
    amax = np.abs(y.reshape(40, 2, 32)).max(axis=2)
    assert np.all(amax <= 448 * s)
    assert np.all((amax > 224 * s) | (s == 2.0 ** -127))
    assert s[1, 0] == 1 and s[2, 0] == 2 and s[0, 0] == 2.0 ** -127


def test_clip():
    rng = np.random.default_rng(3)
    g = [rng.standard_normal(5), rng.standard_normal((2, 3)), np.zeros(0)]
    n, out = tail.grad_clip(g, 1.5)
    assert abs(n - np.linalg.norm(np.concatenate([a.ravel() for a in g]))) < 1e-14
    assert abs(np.linalg.norm(np.concatenate([a.ravel() for a in out])) - 1.5) < 1e-14
    assert all(np.array_equal(a, b) for a, b in zip(tail.grad_clip(g, 1e9)[1], g))


def test_linear_logprob_finite_differences():
    rng = np.random.default_rng(4)
    C, V, D, S, scale = 4, 6, 3, 9, 0.7
    x, w = rng.standard_normal((C, D)), rng.standard_normal((V, D))
    sem_row = np.array([0, 0, 0, 1, 1, 2, 2, 2, 0])      # row 3 has no position
    target = np.array([1, 1, 4, 0, -1, 5, 6, 2, 3])      # -1 and 6 are no labels
    g = rng.standard_normal(S)

    def loss():
        return float((tail.linear_logprob_fwd(x, w, sem_row, target, scale)[0] * g).sum())

    logp, _ = tail.linear_logprob_fwd(x, w, sem_row, target, scale)
    assert logp[4] == 0 and logp[6] == 0 and np.all(logp[[0, 3, 5]] < 0)
    dx, dw = tail.linear_logprob_bwd(x, w, sem_row, target, g, scale)
    np.testing.assert_allclose(dx, _differences(loss, x), atol=1e-7)
    np.testing.assert_allclose(dw, _differences(loss, w), atol=1e-7)
    assert np.all(dx[3] == 0)
