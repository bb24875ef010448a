"""The oracle of the block norms against central differences and hand cases."""
import numpy as np
import pytest

from oracle.block_norm import backward, forward, gate


def test_gates():
    z = np.array([-800.0, -1.0, 0.0, 2.0, 800.0])
    assert np.allclose(gate(z, "sigmoid")[0], [0, 1 / (1 + np.e), 0.5, 1 / (1 + np.exp(-2)), 1])
    assert np.allclose(gate(z, "silu")[0], z * gate(z, "sigmoid")[0])
    assert gate(z, "linear")[0] is z
    for act in ("silu", "sigmoid"):
        assert np.allclose((gate(z + 1e-6, act)[0] - gate(z - 1e-6, act)[0]) / 2e-6, gate(z, act)[1], atol=1e-8)


def test_hand_case():
    y = np.array([[3.0, 4.0]])
    h, n, r1, r2 = forward(y, np.array([1.0, 2.0]), None, "linear", 0.5, np.array([[1.0, -1.0]]), None, 0.0)
    rms = np.sqrt(12.5)
    assert np.allclose(r1, 1 / rms) and np.allclose(h, [[0.5 * 3 / rms + 1, 0.5 * 8 / rms - 1]]) and n is None and r2 is None


@pytest.mark.parametrize("post,g,act,pre", [(1, 1, "silu", 1), (1, 0, "linear", 1), (1, 1, "sigmoid", 0), (0, 1, "linear", 1),
                                            (0, 0, "linear", 1), (1, 1, "linear", 0)])
def test_gradients_against_differences(post, g, act, pre):
    r = np.random.default_rng(post + 2 * g + 4 * pre)
    C, D = 3, 7
    v = {"y": r.standard_normal((C, D)), "post": r.standard_normal(D) if post else None, "g": r.standard_normal((C, D)) if g else None,
         "res": r.standard_normal((C, D)), "pre": r.standard_normal(D) if pre else None}
    dn, dh = r.standard_normal((C, D)), r.standard_normal((C, D))

    def run(v):
        return forward(v["y"], v["post"], v["g"], act, 0.7, v["res"], v["pre"], 1e-3)
    h, _, r1, r2 = run(v)
    # the reciprocal roots hold eps, so the mean of squares in the gradient is the plain formula
    d = backward(v["y"], h, dn if pre else None, dh, v["post"], v["g"], act, 0.7, v["pre"], r1, r2)

    def loss(v):
        h, n, _, _ = run(v)
        return np.sum(h * dh) + (np.sum(n * dn) if pre else 0.0)
    names = {"y": "dy", "res": "dresidual", "g": "dgate", "post": "dpost_weight", "pre": "dpre_weight"}
    for k, name in names.items():
        if v[k] is None:
            continue
        dirn = r.standard_normal(v[k].shape)
        up, down = dict(v), dict(v)
        up[k], down[k] = v[k] + 1e-6 * dirn, v[k] - 1e-6 * dirn
        diff = (loss(up) - loss(down)) / 2e-6
        assert abs(diff - np.sum(d[name] * dirn)) <= 1e-6 * (1 + abs(diff)), name
