"""harts_block_norm_fwd / _bwd at the ends of their ranges."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from prefix_shared_chunkwise_gb300.api import block_norm_bwd
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


# Rows above 4,096 channels: 152 blocks take one row at a time, three or four of them each here, from one stage or two of
# the ring (bf16 with everything: two up to about 7,300 channels), with the weights' gradients in shared memory.
WIDE = [(500, D, "all", dtype) for D in (4104, 5120, 7304, 7328, 8192, 4097, 5001, 8191) for dtype in ("bf16", "fp32")]
WIDE += [(500, D, form, dtype) for D in (5120, 8192, 5001) for form in ("plain", "heads", "bare") for dtype in ("bf16", "fp32")]


@pytest.mark.parametrize("C,D,form,dtype", WIDE)
def test_wide_rows_over_several_passes(C, D, form, dtype):
    c = Case(C, D, dtype, form)
    c.check_backward(*c.check_forward())


SUMS = [(70_001, 128), (2_000_003, 8), (50_003, 3), (40_001, 67), (20_000, 100), (65_536, 512), (9001, 1024), (5000, 2048), (3001, 513),
        (2501, 1025), (1500, 4096), (901, 2047), (900, 8192), (700, 5120), (777, 8189), (700, 5001)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("form", ["block", "head", "pre"])
@pytest.mark.parametrize("C,D", SUMS)
def test_weights_gradients_miss_no_row(C, D, form, gated, dtype):
    """Small whole numbers, reciprocal roots of 1 and a second weight of 0 (which leaves the gradient of h as it
    arrives): every row adds a whole number to either sum, fp32 holds them all, and the sums are exact in any order."""
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(C + D)
    whole = lambda: torch.randint(-2, 3, (C, D), generator=g, device="cuda").to(td)
    post, pre = form != "pre", form != "head"
    y, h, dn, dh, gate = whole(), whole(), whole(), whole(), whole()
    w1, w2, one = torch.ones(D, device="cuda"), torch.zeros(D, device="cuda"), torch.ones(C, device="cuda")
    d = block_norm_bwd(y, h if pre else None, dn if pre else None, dh, post_weight=w1 if post else None, gate=gate if gated else None,
                       gate_act="linear", scale=1.0, pre_weight=w2 if pre else None, rstd_post=one if post else None,
                       rstd_pre=one if pre else None)
    total = lambda *t: torch.stack([v.long() for v in t]).prod(0).sum(0).double()
    if post:
        assert torch.equal(d["dpost_weight"].double(), total(dh, y, gate) if gated else total(dh, y))
    if pre:
        assert torch.equal(d["dpre_weight"].double(), total(dn, h))
        assert torch.equal(d["dresidual"], dh)
