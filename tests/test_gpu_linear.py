"""GPU parity of harts_linear_fwd / _bwd against the fp64 oracle (oracle/linear.py) on the same
(cast) inputs, element by element.

Bounds.  u = 2^-24, r = 2^-8 (a half step of bf16 relative to the value).  A sum of S products is
cut towards zero at most once in 16 of them and once more for each piece it is joined from:
(S/16 + 40) 2 u of the sum of the products' sizes; as dot products, chains of S/32 + 10 roundings.
Both are within (S/8 + 80) u =: k.  silu: sigmoid's exponential, its argument, a sum and a
reciprocal, (10 + 1.5 |z|) u; gelu: 7e-7 of the fit, the exponential's argument z^2 and itself,
(14 + z^2) u; the derivative of either is at most 1.13, which carries z's own error.  The
backward's dz is rounded to bf16 where there is an activation: r |dz| in every product."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytest.importorskip("scipy")

from oracle import linear as ref
from prefix_shared_chunkwise_gb300.api import linear_bwd, linear_fwd

pytestmark = pytest.mark.gpu

U, R = 2.0 ** -24, 2.0 ** -8
# one row and the rows around the dot products' limit, a tile's, a pair's and beyond; widths that are not
# whole panels, narrower than one, of several tiles; long sums over few tiles
SIZES = [(1, 8, 8), (1, 2048, 1000), (2, 264, 8), (3, 72, 136), (5, 1032, 72), (8, 512, 520), (9, 512, 520), (31, 8, 2048),
         (64, 2048, 64), (100, 136, 264), (128, 64, 256), (129, 192, 200), (256, 4096, 128), (257, 72, 8), (300, 1032, 1000),
         (777, 2760, 1032), (1000, 40, 56), (2049, 512, 384), (5000, 128, 136)]


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from prefix_shared_chunkwise_gb300 import build
    build.build()


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _gate_error(z, kind):
    """What the activation's factor of z (or its slope) is off by, relative to 1 + |z|."""
    if kind == "none":
        return 0.0
    return (12 + 2 * np.abs(z)) * U if kind == "silu" else 7e-7 + (16 + z * z) * U


class Case:
    def __init__(self, C, K, N, bias, res, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed + C + K + N)
        rand = lambda *s: torch.randn(s, generator=g, device="cuda")
        self.x, self.w = rand(C, K).bfloat16(), (2 * rand(N, K) / K ** 0.5).bfloat16()
        self.b = rand(N) if bias else None
        self.res = rand(C, N).bfloat16() if res else None
        self.dy = rand(C, N).bfloat16()
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def check_forward(self, kind, keep):
        y, z = linear_fwd(self.x, self.w, self.b, self.res, activation=kind, keep_z=keep, error=self.err)
        torch.cuda.synchronize()
        assert int(self.err) == 0
        x, w, b, res = map(_np, (self.x, self.w, self.b, self.res))
        ry, rz = ref.forward(x, w, b, res, kind)
        k = (x.shape[1] / 8 + 80) * U
        e = k * (np.abs(x) @ np.abs(w).T) + U * np.abs(rz)
        if keep:
            assert np.all(np.abs(_np(z) - rz) <= R * np.abs(rz) + e + 1e-37)
        else:
            assert z is None
        body = ry - (0.0 if res is None else res)
        bound = R * np.abs(ry) + 1.13 * e + _gate_error(rz, kind) * np.abs(body) + 2 * U * (np.abs(ry) + np.abs(body))
        assert np.all(np.abs(_np(y) - ry) <= bound + 1e-37)
        return y, z

    def check_backward(self, kind, z, with_bias):
        got = linear_bwd(self.x, self.w, self.dy, z, activation=kind, with_bias=with_bias, error=self.err)
        torch.cuda.synchronize()
        assert int(self.err) == 0
        x, w, dy, zn = map(_np, (self.x, self.w, self.dy, z))
        rdx, rdw, rdb, dz = ref.backward(x, w, dy, zn, kind)
        e = 0.0 if kind == "none" else np.abs(dy) * _gate_error(zn, kind) * (1 + np.abs(zn)) + U * np.abs(dz)
        size = np.abs(dz) + e
        held = e + (0.0 if kind == "none" else R * size)
        for out, want, a, b, s in ((got[0], rdx, np.asarray(size), np.abs(w), w.shape[0]), (got[1], rdw, np.asarray(size).T, np.abs(x), len(x))):
            h = held if np.isscalar(held) else (held if a is size else held.T)
            bound = R * np.abs(want) + (s / 8 + 80) * U * ((a + h) @ b) + (0.0 if np.isscalar(h) else h @ b)
            assert np.all(np.abs(_np(out) - want) <= bound + 1e-37)
        if with_bias:
            total = np.sum(size, axis=0)
            assert np.all(np.abs(_np(got[2]) - rdb) <= (len(x) / 32 + 80) * U * total + (0.0 if kind == "none" else np.sum(e, axis=0)) + 1e-37)
        else:
            assert got[2] is None
        again = linear_bwd(self.x, self.w, self.dy, z, activation=kind, with_bias=with_bias)
        assert all(torch.equal(a, b) for a, b in zip(got, again) if a is not None)


@pytest.mark.parametrize("kind,bias,res,keep", [("none", False, False, False), ("gelu", True, True, True), ("silu", True, False, True),
                                                ("none", True, True, True), ("gelu", False, True, False)])
@pytest.mark.parametrize("C,K,N", SIZES)
def test_forward(C, K, N, kind, bias, res, keep):
    Case(C, K, N, bias, res).check_forward(kind, keep)


@pytest.mark.parametrize("kind,bias", [("none", False), ("gelu", True), ("silu", False), ("none", True)])
@pytest.mark.parametrize("C,K,N", SIZES)
def test_backward(C, K, N, kind, bias):
    c = Case(C, K, N, bias, False)
    _, z = linear_fwd(c.x, c.w, c.b, activation=kind, keep_z=kind != "none")
    c.check_backward(kind, z, bias)


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_far_out(kind):
    """Values from the far tails to where the activation is the identity."""
    c = Case(300, 64, 128, True, False)
    c.w *= 0
    c.b.copy_(torch.linspace(-30, 30, 128))
    y, z = c.check_forward(kind, True)
    c.check_backward(kind, z, True)
    assert bool(y.isfinite().all())
    one = linear_fwd(c.x[:3].contiguous(), c.w, c.b, activation=kind)[0]      # as dot products
    assert torch.equal(one, y[:3])


def test_rows_do_not_reach_one_another():
    c = Case(300, 256, 136, True, True)
    y, z = linear_fwd(c.x, c.w, c.b, c.res, activation="gelu", keep_z=True)
    c.x[200, 7] = float("nan")
    c.res[100, 3] = float("inf")
    y2, z2 = linear_fwd(c.x, c.w, c.b, c.res, activation="gelu", keep_z=True)
    rows = [i for i in range(300) if i not in (100, 200)]
    assert torch.equal(y[rows], y2[rows]) and torch.equal(z[rows], z2[rows])
    assert bool(y2[200].isnan().all()) and torch.equal(z2[100], z[100])
    assert bool(y2[100, 3].isinf()) and torch.equal(y2[100, 4:], y[100, 4:])


@pytest.mark.parametrize("C", [5, 100, 2000])
def test_in_place_and_given_buffers(C):
    c = Case(C, 520, 264, True, True)
    y, _ = linear_fwd(c.x, c.w, c.b, c.res, activation="silu")
    res = c.res.clone()
    got, _ = linear_fwd(c.x, c.w, c.b, res, activation="silu", y=res)
    assert got is res and torch.equal(got, y)
    # what lies behind a buffer stays as it is
    big = torch.full((C + 8, 264), 7.0, dtype=torch.bfloat16, device="cuda")
    linear_fwd(c.x, c.w, c.b, c.res, activation="silu", y=big[:C])
    assert torch.equal(big[:C], y) and bool((big[C:] == 7).all())
    bx = torch.full((C + 8, 520), 7.0, dtype=torch.bfloat16, device="cuda")
    bw = torch.full((272, 520), 7.0, dtype=torch.bfloat16, device="cuda")
    dx, dw, _ = linear_bwd(c.x, c.w, c.dy)
    linear_bwd(c.x, c.w, c.dy, dx=bx[:C], dweight=bw[:264])
    assert torch.equal(bx[:C], dx) and torch.equal(bw[:264], dw)
    assert bool((bx[C:] == 7).all()) and bool((bw[264:] == 7).all())


def test_captured_and_on_another_stream():
    for C in (4, 200, 3000):
        c = Case(C, 512, 768, True, True)

        def run(**kw):
            y, z = linear_fwd(c.x, c.w, c.b, c.res, activation="gelu", keep_z=True, **kw)
            return [y, z, *linear_bwd(c.x, c.w, c.dy, z, activation="gelu", with_bias=True, **kw)]
        want = run()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        got = run(stream=s)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = run()
        for _ in range(2):
            for t in got:
                t.zero_()
            graph.replay()
            assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_no_rows():
    x, w = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), torch.ones((16, 64), dtype=torch.bfloat16, device="cuda")
    y, z = linear_fwd(x, w, activation="gelu", keep_z=True)
    assert y.shape == z.shape == (0, 16)
    dx, dw, db = linear_bwd(x, w, y, z, activation="gelu", with_bias=True)
    assert dx.shape == (0, 64) and bool((dw == 0).all()) and bool((db == 0).all())
