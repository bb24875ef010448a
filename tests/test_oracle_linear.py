"""The projection's oracle against hand values and central differences."""
import numpy as np
import pytest

pytest.importorskip("scipy")

from oracle.linear import act, backward, forward


def test_activations():
    z = np.array([-40.0, -1.0, 0.0, 1.0, 40.0])
    assert np.allclose(act(z, "gelu")[0], [0, -0.15865525393145707, 0, 0.8413447460685429, 40])
    assert np.allclose(act(z, "silu")[0], [0, -1 / (1 + np.e), 0, np.e / (1 + np.e), 40])
    for kind in ("none", "silu", "gelu"):
        assert np.allclose((act(z + 1e-6, kind)[0] - act(z - 1e-6, kind)[0]) / 2e-6, act(z, kind)[1], atol=1e-8)


@pytest.mark.parametrize("kind", ["none", "silu", "gelu"])
def test_gradients_against_differences(kind):
    r = np.random.default_rng(1)
    x, w, b, res, dy = (r.standard_normal(s) for s in ((5, 4), (3, 4), 3, (5, 3), (5, 3)))
    y, z = forward(x, w, b, res, kind)
    dx, dw, db, _ = backward(x, w, dy, z, kind)
    for i, g in ((0, dx), (1, dw), (2, db), (3, dy)):
        d = r.standard_normal(g.shape)
        up, down = [x, w, b, res], [x, w, b, res]
        up[i], down[i] = up[i] + 1e-6 * d, down[i] - 1e-6 * d
        diff = np.sum((forward(*up, kind)[0] - forward(*down, kind)[0]) * dy) / 2e-6
        assert abs(diff - np.sum(g * d)) <= 1e-7 * (1 + abs(diff))
