"""harts_scan_fwd / _bwd at the ends of their ranges.  u = 2^-24."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from prefix_shared_chunkwise_gb300.api import Plan, scan_bwd, scan_fwd
from tests.test_gpu_scan import FORESTS, LONG, Case

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from prefix_shared_chunkwise_gb300 import build
    build.build()


@pytest.mark.parametrize("rows", [1, 2])
def test_decays_from_the_smallest_to_the_largest(rows):
    """What a decay and its complement are themselves: h = a (x = 0, h0 = 1), h = 1 - a (x = 1, h0 = 0), dx = (1 - a)
    dh and dg = a dh (h0 = 1, x = 0), in roots of one row (a decoding step's kernel) and of two (the tiles').
    f = g log2 e - n has two roundings of at most 2^-26, 0.35 u of a in all; t = 2^f - 1 is off by f's share
    and five half steps of the last terms of its series, less than 3 u of |t| <= 0.42; a = scale (1 + t) rounds once more: 0.35 +
    1.3 + 0.5 < 2.5 u.  1 - a is t itself near a = 1: 3.5 u with f's two roundings relative to f.  The mix form's forward
    has a from 1 - a, 2^-25 + 3.5 u of 1 - a off; results below fp32's normal range count as 2^-126."""
    B, D = 64, 512
    g = -torch.logspace(-7, np.log10(87.0), B * D, dtype=torch.float64).float().view(B, 1, D)
    g = torch.cat([g, torch.full((B, rows - 1, D), -1.0)], dim=1).reshape(B * rows, D).cuda()
    plan = Plan([-1] * B, [rows] * B, 64).upload()
    first = torch.arange(B, device="cuda") * rows
    g64 = g[first].double().cpu().numpy()
    a, rest = np.exp(g64), -np.expm1(g64)
    one, zero, h0 = torch.ones_like(g), torch.zeros_like(g), torch.ones(B, D, device="cuda")
    got = lambda t: t[first].double().cpu().numpy()
    tiny = 2.0 ** -126
    h = scan_fwd(plan, zero, g, h0=h0)
    assert np.all(np.abs(got(h) - a) <= 2.5 * U * a + tiny)
    assert np.all(np.abs(got(scan_fwd(plan, one, g, form="mix")) - rest) <= 3.5 * U * rest)
    assert np.all(np.abs(got(scan_fwd(plan, zero, g, form="mix", h0=h0)) - a) <= 2.0 ** -25 + 3.5 * U * rest + U * a)
    dh = torch.zeros_like(g)
    dh[first] = 1.0
    for form in ("add", "mix"):
        dx, dg = scan_bwd(plan, zero, g, h, dh, form=form, h0=h0)
        assert np.all(np.abs(got(dx) - (rest if form == "mix" else 1.0)) <= (3.5 * U * rest if form == "mix" else 0.0))
        assert np.all(np.abs(got(dg) - a) <= 2.5 * U * a + U * a + tiny)
    torch.cuda.synchronize()
    assert plan.device_error() == 0


@pytest.mark.parametrize("form,state", [("add", False), ("mix", True), ("add", True)])
@pytest.mark.parametrize("forest", ["groups", "group-ends", "trees", "forks"])
def test_groups_of_eight_tiles(forest, form, state):
    """More than 512 bf16 channels, whose forward joins eight tiles' maps at most, against the oracle."""
    c = Case({**FORESTS, **LONG}[forest], 1000, "bf16", form, state, seed=2)
    c.check_backward(c.check_forward())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("children", [64, 513])
def test_many_branches_of_one_segment(children, dtype):
    """The gradient behind a wide fork is a sum over all its branches, by ascending segment."""
    c = Case(([-1] + [0] * children, [300] + [1 + (11 * i) % 40 for i in range(children)]), 72, dtype, "mix", True, seed=3)
    c.check_backward(c.check_forward())


@pytest.mark.parametrize("forest", ["steps", "trees"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_states_and_their_gradients_one_without_the_other(forest, dtype):
    """No h0 is an h0 of zeros, no d_final a d_final of zeros, and what is not asked for changes nothing else."""
    c = Case(FORESTS[forest], 72, dtype, "mix", True, seed=4)
    c.h0.zero_()
    c.dfinal.zero_()
    h, final = c.forward()
    assert torch.equal(scan_fwd(c.plan, c.x, c.g, form="mix"), h)
    got = torch.full_like(final, 7.0)
    scan_fwd(c.plan, c.x, c.g, form="mix", final_state=got)
    assert torch.equal(got, final)
    dx, dg, dh0 = c.backward(h)
    for kw in ({}, {"h0": c.h0}, {"d_final": c.dfinal}):
        got = torch.full_like(dh0, 7.0)
        out = scan_bwd(c.plan, c.x, c.g, h, c.dh, form="mix", dh0=got, **kw)
        assert torch.equal(out[0], dx) and torch.equal(out[1], dg) and torch.equal(got, dh0)
        assert all(torch.equal(a, b) for a, b in zip(scan_bwd(c.plan, c.x, c.g, h, c.dh, form="mix", **kw), (dx, dg)))
