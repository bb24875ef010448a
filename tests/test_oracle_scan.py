"""The oracle of the gated recurrence against something other than itself: closed forms, the same
rows over every trajectory alone, and central differences."""
import numpy as np
import pytest

from oracle.scan import scan_forest, scan_forest_bwd

PARENT = [-1, 0, 0, 2, -1, 2, 5]
LEN = [4, 3, 1, 5, 2, 3, 1]
OFF = [0, 4, 12, 13, 7, 9, 18]                  # in no particular order


def _case(seed, D=3):
    r = np.random.default_rng(seed)
    C = sum(LEN)
    x, dh = r.standard_normal((C, D)), r.standard_normal((C, D))
    return r, x, -np.abs(r.standard_normal((C, D))), dh, r.standard_normal((2, D))


def test_closed_forms():
    x = np.ones((6, 2))
    h, prev = scan_forest([-1], [6], [0], x, np.full((6, 2), np.log(0.5)), False)
    assert np.allclose(h[:, 0], 2 - 0.5 ** np.arange(6)) and np.all(prev[1:] == h[:-1]) and np.all(prev[0] == 0)
    h, _ = scan_forest([-1], [6], [0], x, np.full((6, 2), np.log(0.25)), True, h0=np.ones((1, 2)))
    assert np.allclose(h, 1)                    # a mean of ones
    h, _ = scan_forest([-1], [6], [0], x, np.full((6, 2), -np.inf), False)
    assert np.array_equal(h, x)                 # everything forgotten
    h, _ = scan_forest([-1], [6], [0], x, np.zeros((6, 2)), False)
    assert np.allclose(h[:, 1], np.arange(1, 7))


@pytest.mark.parametrize("mix", [False, True])
def test_equal_to_every_trajectory_alone(mix):
    _, x, g, _, h0 = _case(1)
    h, _ = scan_forest(PARENT, LEN, OFF, x, g, mix, h0)
    for leaf in (1, 3, 4, 6):
        chain, v = [], leaf
        while v >= 0:
            chain.insert(0, v)
            v = PARENT[v]
        rows = np.concatenate([np.arange(OFF[v], OFF[v] + LEN[v]) for v in chain])
        alone, _ = scan_forest([-1], [len(rows)], [0], x[rows], g[rows], mix, h0[[0 if chain[0] == 0 else 1]])
        assert np.array_equal(alone, h[rows])


@pytest.mark.parametrize("mix", [False, True])
def test_gradients_against_differences(mix):
    r, x, g, dh, h0 = _case(2)
    ends = {OFF[v] + LEN[v] - 1: r.standard_normal(3) for v in (1, 3, 4, 6)}
    _, prev = scan_forest(PARENT, LEN, OFF, x, g, mix, h0)
    dx, dg, dh0, _ = scan_forest_bwd(PARENT, LEN, OFF, x, g, mix, prev, dh, h0, ends)

    def loss(x, g, h0):
        h, _ = scan_forest(PARENT, LEN, OFF, x, g, mix, h0)
        return np.sum(h * dh) + sum(np.sum(h[r_] * d) for r_, d in ends.items())
    for i, grad in enumerate((dx, dg, dh0)):
        dirn = r.standard_normal(grad.shape)
        args = [x, g, h0]
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + 1e-6 * dirn, args[i] - 1e-6 * dirn
        diff = (loss(*up) - loss(*down)) / 2e-6
        assert abs(diff - np.sum(grad * dirn)) <= 1e-7 * (1 + abs(diff))
