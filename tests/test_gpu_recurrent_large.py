"""Tensors of more than 2^31 values: the last rows come out with the bits that they have in a call of their own."""
import pytest

torch = pytest.importorskip("torch")

from prefix_shared_chunkwise_gb300.api import (Plan, block_norm_bwd, block_norm_fwd, linear_bwd, linear_fwd, scan_bwd,
                                               scan_fwd)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from prefix_shared_chunkwise_gb300 import build
    build.build()


@pytest.fixture(autouse=True)
def emptied():
    yield
    torch.cuda.empty_cache()


def _rand(seed, *shape):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda", dtype=torch.bfloat16)


@pytest.mark.parametrize("form", ["add", "mix"])
def test_scan(form):
    D, length = 4096, [300, 128, 4000, 77]                   # two trees of a branch each, over and over
    n = (2 ** 31 // D) // sum(length) + 1
    parent = [q for i in range(n) for q in (-1, 4 * i, -1, 4 * i + 2)]
    large, small = Plan(parent, length * n, 64).upload(), Plan(parent[:4], length, 64).upload()
    offs, off = (p.arrays()["seg_offset"] for p in (large, small))
    C, c = large.info["C"], small.info["C"]
    assert C * D > 2 ** 31
    rows = torch.cat([torch.arange(int(o), int(o) + k) for o, k in zip(offs[-4:], length)]).cuda()
    own = torch.cat([torch.arange(int(o), int(o) + k) for o, k in zip(off, length)]).cuda()
    x, dh = _rand(1, C, D), _rand(2, C, D)
    g = _rand(3, C, D).abs_().neg_()
    cut = lambda t: torch.empty((c, D), dtype=t.dtype, device="cuda").index_copy_(0, own, t[rows])
    h = scan_fwd(large, x, g, form=form)
    h2 = scan_fwd(small, cut(x), cut(g), form=form)
    assert torch.equal(cut(h), h2)
    d, d2 = scan_bwd(large, x, g, h, dh, form=form), scan_bwd(small, cut(x), cut(g), h2, cut(dh), form=form)
    assert large.device_error() == small.device_error() == 0
    assert all(torch.equal(cut(a), b) for a, b in zip(d, d2))


@pytest.mark.parametrize("D", [2048, 2001])
def test_block_norm(D):
    C, last = 2 ** 31 // D + 1001, 1000
    last -= (C - last) % 2                                   # rows of odd width begin as they do there
    t = {k: _rand(i, C, D) for i, k in enumerate(("y", "gate", "residual", "dn", "dh"))}
    w = torch.rand(D, device="cuda") + 0.5

    def run(t):
        kw = dict(post_weight=w, gate=t["gate"], pre_weight=w)
        h, n, r1, r2 = block_norm_fwd(t["y"], residual=t["residual"], **kw)
        d = block_norm_bwd(t["y"], h, t["dn"], t["dh"], rstd_post=r1, rstd_pre=r2, **kw)
        return h, n, r1, r2, d["dy"], d["dresidual"], d["dgate"]
    for a, b in zip(run(t), run({k: v[-last:].clone() for k, v in t.items()})):
        assert torch.equal(a[-last:], b)


def test_linear():
    K, N = 64, 8192
    C, last = 2 ** 31 // N + 2057, 5000                      # the same rule cuts either into whole sums
    x, w, dy, b = _rand(1, C, K), _rand(2, N, K), _rand(3, C, N), torch.randn(N, device="cuda")

    y, z = linear_fwd(x, w, b, dy, activation="silu", keep_z=True)
    y2, z2 = linear_fwd(x[-last:].clone(), w, b, dy[-last:].clone(), activation="silu", keep_z=True)
    assert torch.equal(y[-last:], y2) and torch.equal(z[-last:], z2)
    dx = linear_bwd(x, w, dy, z, activation="silu")[0][-300:].double()
    z, dy = z[-300:].double(), dy[-300:].double()
    q = torch.sigmoid(z)
    dz = dy * q * (1 + z * (1 - q))
    want, size = dz @ w.double(), dz.abs() @ w.double().abs()
    assert bool(((dx - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -13) * size).all())      # dz rounded, then dx


def test_linear_by_a_wide_sum():
    """More than 2^31 values of x: dx, and dweight over all of them by a gradient that is zero but in the last rows."""
    K, N = 8192, 72
    C, last = 2 ** 31 // K + 2057, 300
    x, w, dy = _rand(1, C, K), _rand(2, N, K), torch.zeros((C, N), dtype=torch.bfloat16, device="cuda")
    dy[-last:] = _rand(3, last, N)
    dx, dw, db = linear_bwd(x, w, dy, with_bias=True)
    assert bool((dx[:-last] == 0).all())
    x, dy = x[-last:].double(), dy[-last:].double()
    size = dy.abs().T @ x.abs()
    assert bool(((dw.double() - dy.T @ x).abs() <= 2.0 ** -8 * (dy.T @ x).abs() + 2.0 ** -17 * size).all())
    assert bool(((dx[-last:].double() - dy @ w.double()).abs() <= 2.0 ** -8 * (dy @ w.double()).abs() + 2.0 ** -17 * (dy.abs() @ w.double().abs())).all())
    assert bool(((db.double() - dy.sum(0)).abs() <= 2.0 ** -20 * dy.abs().sum(0)).all())
