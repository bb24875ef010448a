"""GPU parity of harts_rmsnorm_fwd / _bwd against the fp64 oracle (oracle/tail.py) on the same
(cast) inputs, element by element.

Bounds.  u = 2^-24 (fp32 half step), r = half a step of the output type relative to the value
(bf16 2^-8, fp32 u).  A row's sum of squares of D values in chains of at most D/32 + 10
additions is off by that many u, its square root by half of it; y adds the rounding of h, rstd
and two products: |y - ref| <= (r + (D/64 + 12) u) |ref| up to the type's smallest step.
dx is a difference of terms t = |rstd w dy| and |n| mean|w dy n|, plus dh: each within
(D/32 + 16) u of itself, and one rounding.  dweight sums C products in fp32 chains of at most
C + 16 additions.  8-bit: half a step of a 4-bit significand, 2^-4 of the value, or half of
the smallest step 2^-9 of the scale; the scale is compared with its definition."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import tail
from prefix_shared_chunkwise_gb300.api import rmsnorm_bwd, rmsnorm_fwd

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": (torch.bfloat16, 2.0 ** -8), "fp32": (torch.float32, U)}
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from prefix_shared_chunkwise_gb300 import build
    build.build()


def _rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _np(t):
    return t.double().cpu().numpy()


def _check_fwd(x, res, w, dtype, eps=EPS):
    td, r = DT[dtype]
    y, h, rstd = rmsnorm_fwd(x, w, res, eps=eps)
    torch.cuda.synchronize()
    ry, rh, rr = tail.rmsnorm_fwd(_np(x), None if res is None else _np(res), _np(w), eps)
    D = x.shape[1]
    k = (D / 64 + 12) * U
    assert np.all(np.abs(_np(h) - rh) <= r * np.abs(rh) + 1e-38)
    assert np.all(np.abs(_np(rstd) - rr) <= k * rr)
    assert np.all(np.abs(_np(y) - ry) <= (r + k) * np.abs(ry) + 1e-38), np.max(np.abs(_np(y) - ry) / np.abs(ry).max())
    if res is None:
        assert h is x
    return y, h, rstd


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("C,D", [(1, 1), (1, 8), (3, 7), (5, 32), (1, 2048), (700, 64), (33, 1000), (129, 1001),
                                 (37, 4096), (6, 8192), (3, 8191), (3, 16384), (2, 16383), (2000, 264)])
def test_forward(dtype, C, D):
    td, _ = DT[dtype]
    w = _rand((D,), torch.float32, 3)
    _check_fwd(_rand((C, D), td, 1), _rand((C, D), td, 2, 3.0), w, dtype)
    _check_fwd(_rand((C, D), td, 4, 1e-3), None, w, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("C,D", [(1, 1), (3, 7), (1, 2048), (700, 64), (1237, 1001), (5000, 256), (37, 4096),
                                 (3, 8191), (3, 16384), (2, 16383), (40000, 128)])
def test_backward(dtype, residual, C, D):
    td, r = DT[dtype]
    dy, h, w = _rand((C, D), td, 1), _rand((C, D), td, 2, 2.0), _rand((D,), torch.float32, 3)
    dh = _rand((C, D), td, 4) if residual else None
    rstd = torch.rsqrt(h.double().square().mean(1) + EPS).float()
    dx, dw = rmsnorm_bwd(dy, h, w, rstd, dh)
    torch.cuda.synchronize()
    rdx, rdw = tail.rmsnorm_bwd(_np(dy), _np(h), _np(w), _np(rstd), None if dh is None else _np(dh))
    rs = _np(rstd)[:, None]
    n, t = _np(h) * rs, _np(dy) * _np(w)
    size = rs * (np.abs(t) + np.abs(n) * np.abs(t * n).mean(axis=1, keepdims=True))
    if dh is not None:
        size = size + np.abs(_np(dh))
    assert np.all(np.abs(_np(dx) - rdx) <= r * np.abs(rdx) + (D / 32 + 16) * U * size)
    assert np.all(np.abs(_np(dw) - rdw) <= (C + 16) * U * np.abs(_np(dy) * n).sum(axis=0))
    dx2, dw2 = rmsnorm_bwd(dy, h, w, rstd, dh)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)          # no order of additions left open


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("C,D", [(1, 64), (7, 40), (33, 64), (1000, 128), (129, 96), (5, 256), (1003, 200), (77, 512),
                                 (2, 2048), (500, 2048), (9, 4096), (5, 8192), (3, 12288), (6, 9000)])
def test_short_and_long_rows(dtype, C, D):
    """Several rows a warp or a block, rows copied ahead, rows read twice; C below and above
    what a block works on at a time."""
    td, r = DT[dtype]
    x, res, w = _rand((C, D), td, 1), _rand((C, D), td, 2), _rand((D,), torch.float32, 3)
    _, h, rstd = _check_fwd(x, res, w, dtype)
    dy, dh = _rand((C, D), td, 4), _rand((C, D), td, 5)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for d in (None, dh):
        dx, dw = rmsnorm_bwd(dy, h, w, rstd, d, error=err)
        torch.cuda.synchronize()
        rdx, rdw = tail.rmsnorm_bwd(_np(dy), _np(h), _np(w), _np(rstd), None if d is None else _np(d))
        rs = _np(rstd)[:, None]
        n, t = _np(h) * rs, _np(dy) * _np(w)
        size = rs * (np.abs(t) + np.abs(n) * np.abs(t * n).mean(axis=1, keepdims=True)) + (0 if d is None else np.abs(_np(d)))
        assert np.all(np.abs(_np(dx) - rdx) <= r * np.abs(rdx) + (D / 32 + 16) * U * size)
        assert np.all(np.abs(_np(dw) - rdw) <= (C + 16) * U * np.abs(_np(dy) * n).sum(axis=0))
    assert int(err) == 0


def test_backward_against_differences():
    """dL/dx of L = <y, dy> + <h, dh> in fp32 against central differences of the forward
    kernel along one direction.  Step 2^-6: the third-order term is about rstd^2 step^2 / 2, 6e-5,
    of the terms; the fp32 rounding of the 2,000 outputs adds ~2^-24 * 45 / step, 1e-7 of
    their sum."""
    C, D, step = 4, 500, 2.0 ** -6
    x, r, w = _rand((C, D), torch.float32, 1), _rand((C, D), torch.float32, 2), _rand((D,), torch.float32, 3)
    dy, dh, v = (_rand((C, D), torch.float32, s) for s in (4, 5, 6))

    def loss(a):
        y, h, _ = rmsnorm_fwd(a, w, r, eps=EPS)
        return float((y.double() * dy.double()).sum() + (h.double() * dh.double()).sum())

    _, h, rstd = rmsnorm_fwd(x, w, r, eps=EPS)
    dx, _ = rmsnorm_bwd(dy, h, w, rstd, dh)
    got = float((dx.double() * v.double()).sum())
    num = (loss(x + step * v) - loss(x - step * v)) / (2 * step)
    assert abs(got - num) <= 1e-4 * float((dx.double() * v.double()).abs().sum())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("C,D", [(1, 32), (3, 2048), (257, 96), (19, 4096), (2, 16384)])
def test_mx8(dtype, C, D):
    td, _ = DT[dtype]
    x, res = _rand((C, D), td, 1), _rand((C, D), td, 2)
    w = _rand((D,), torch.float32, 3) * torch.exp(4 * _rand((D,), torch.float32, 5))
    if C > 2:
        x[1], res[1] = 0, 0                                        # a row of zeros
    (q, s), h, rstd = rmsnorm_fwd(x, w, res, eps=EPS, mx8=True)
    y, _, _ = rmsnorm_fwd(x, w, res, eps=EPS)
    torch.cuda.synchronize()
    ry, _, _ = tail.rmsnorm_fwd(_np(x), _np(res), _np(w), EPS)
    scale = _np(s.float())
    want = tail.mx_scales(ry)
    # the kernel's own fp32 y decides; it may fall on the other side of a power of two only
    # where the block's largest value lies within the fp32 error of one
    amax = np.abs(ry.reshape(C, -1, 32)).max(axis=2)
    k = (D / 64 + 12) * U
    assert np.all((scale == want) | (np.abs(amax / 448 / np.minimum(scale, want) - 1) <= 2 * k))
    got = _np(q.float()).reshape(C, -1, 32) * scale[:, :, None]
    ref = ry.reshape(C, -1, 32)
    assert np.all(np.abs(got - ref) <= (2.0 ** -4 + k) * np.abs(ref) + 2.0 ** -10 * scale[:, :, None])
    assert np.all(np.abs(_np(q.float())) <= 448)


def test_not_finite_values_stay_visible():
    D = 128
    x, w = _rand((4, D), torch.bfloat16, 1), torch.ones(D, device="cuda")
    x[1, 5], x[2, 70] = float("nan"), float("inf")
    y, _, rstd = rmsnorm_fwd(x, w)
    (q, s), _, _ = rmsnorm_fwd(x, w, mx8=True)
    torch.cuda.synchronize()
    assert torch.isfinite(y[0]).all() and torch.isfinite(y[3]).all()
    assert torch.isnan(y[1]).all() and torch.isnan(rstd[1])
    assert torch.isnan(y[2, 70]) and float(rstd[2]) == 0
    v = q.float().view(4, -1, 32) * s.float()[:, :, None]
    assert torch.isfinite(v[0]).all() and torch.isnan(v[1]).all() and torch.isnan(v[2].view(-1)[70])


def test_no_rows_and_in_place_and_stream():
    w = torch.ones(64, device="cuda")
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    y, h, rstd = rmsnorm_fwd(e, w, e)
    dx, dw = rmsnorm_bwd(e, e, w, rstd)
    assert y.shape == (0, 64) and dx.shape == (0, 64) and torch.equal(dw, torch.zeros_like(w))
    x, r = _rand((300, 2048), torch.bfloat16, 1), _rand((300, 2048), torch.bfloat16, 2)
    w = _rand((2048,), torch.float32, 3)
    y, h, rstd = rmsnorm_fwd(x, w, r)
    r2, x2 = r.clone(), x.clone()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    y2, h2, _ = rmsnorm_fwd(x2, w, r2, h=r2, y=x2, stream=st)      # h over the residual, y over x
    st.synchronize()
    assert torch.equal(y, y2) and torch.equal(h, h2) and h2 is r2
    d, dh = _rand((300, 2048), torch.bfloat16, 5), _rand((300, 2048), torch.bfloat16, 6)
    dx, dw = rmsnorm_bwd(d, h, w, rstd, dh)
    dx2, dw2 = rmsnorm_bwd(d, h, w, rstd, dh, dx=dh)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_h_without_a_residual(dtype):
    """A given h receives x, and is what the call returns: the backward of a norm in place (y over
    x) is then the one of a norm that kept x."""
    td, _ = DT[dtype]
    x, w, dy = _rand((37, 264), td, 1), _rand((264,), torch.float32, 2), _rand((37, 264), td, 3)
    y, h, rstd = rmsnorm_fwd(x, w)
    assert h is x
    want = rmsnorm_bwd(dy, h, w, rstd)
    own, keep = x.clone(), torch.full_like(x, 7)
    y2, h2, rstd2 = rmsnorm_fwd(own, w, h=keep, y=own)
    torch.cuda.synchronize()
    assert h2 is keep and torch.equal(keep, x) and torch.equal(y2, y) and y2 is own
    got = rmsnorm_bwd(dy, h2, w, rstd2)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    (q, s), h3, _ = rmsnorm_fwd(x[:, :256].contiguous(), w[:256].contiguous(), mx8=True, h=keep[:, :256].contiguous())
    assert torch.equal(h3, x[:, :256])
    inplace = x.clone()
    y4, h4, _ = rmsnorm_fwd(inplace, w, y=inplace)                  # nothing left to differentiate from
    assert h4 is None and torch.equal(y4, y)
    with pytest.raises(RuntimeError, match="one buffer"):
        rmsnorm_fwd(x, w, keep, h=own, y=own)
    none = x[:0]
    assert rmsnorm_fwd(none, w)[1] is none
