"""harts_block_norm_fwd / _bwd at the ends of their ranges."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_block_norm import Case, _np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from prefix_shared_chunkwise_gb300 import build
    build.build()


@pytest.mark.parametrize("D", [512, 131])
@pytest.mark.parametrize("form", ["all", "heads", "pre"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gates_to_the_ends_of_the_type(dtype, form, D):
    """Closed gates are closed however far out they lie: sigmoid is zero there, and so is z sigmoid(z), whose z
    may be 3e38."""
    c = Case(9, D, dtype, form)
    for i, z in enumerate((-80.0, -87.0, -88.0, -89.0, -200.0, -1e30, -3e38, 90.0)):
        c.gate[i] = z
    if form != "heads":                                        # z itself is a factor: keep the block in range
        c.y[7] *= 0.01
    h, r1, r2 = c.check_forward()
    d = c.backward(h, r1, r2)
    torch.cuda.synchronize()
    block = _np(h) - (0.0 if c.res is None else _np(c.res))
    assert np.all(block[4:7] == 0)
    assert bool((d["dgate"][4:7] == 0).all()) and bool((d["dy"][4:7] == 0).all())


@pytest.mark.parametrize("D", [512, 131])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_infinite_gates(dtype, D):
    """sigmoid(-inf) is zero and sigmoid(inf) one; z sigmoid(z) at -inf is no number, as infinity times zero is none."""
    c = Case(6, D, dtype, "heads")
    c.gate[1], c.gate[2] = -torch.inf, torch.inf
    h, _, r1, r2 = c.forward()
    d = c.backward(h, r1, r2)
    assert bool((h[1] == 0).all()) and bool(h[2].isfinite().all()) and bool((d["dgate"][1:3] == 0).all())
    assert bool((d["dy"][1] == 0).all())
    s = Case(6, D, dtype, "all")
    s.gate[1] = -torch.inf
    h = s.forward()[0]
    assert bool(h[1].isnan().all()) and bool(h[[0, 2, 3, 4, 5]].isfinite().all())
