"""GPU parity of harts_block_norm_fwd / _bwd against the fp64 oracle (oracle/block_norm.py) on the
same (cast) inputs, element by element.

Bounds.  u = 2^-24, r half a step of the output type relative to the value (bf16 2^-8, fp32 u).  A
row's sum of D squares, in chains of at most D/32 + 10 additions, leaves its reciprocal root off by
k = (D/64 + 12) u of itself.  sigmoid: the exponential's 2^-22 and its argument's rounding, 4 u +
1.5 |z| u, one addition and a division of 4 u: q is off by (10 + 1.5 |z|) u of itself.  h is then off
by (k + (16 + 1.5 |z|) u) of the gated block, and u of it and the residual; n by that through its own
root.  The backward's rows are differences of terms like rmsnorm's, (D/32 + 20) u of their sizes, and
what the gate's value (as above) and slope ((12 + 2 |z|) u of q (1 + |z|)) are off by; weights'
gradients are fp32 sums in chains of at most C + 20 additions."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import block_norm as ref
from prefix_shared_chunkwise_gb300.api import block_norm_bwd, block_norm_fwd

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": (torch.bfloat16, 2.0 ** -8), "fp32": (torch.float32, U)}
EPS = 1e-6
# post, gate, residual, pre
FORMS = {"all": (1, "silu", 1, 1), "heads": (1, "sigmoid", 0, 0), "plain": (1, None, 1, 1), "post": (1, "linear", 1, 0),
         "pre": (0, "silu", 1, 1), "bare": (0, None, 0, 1)}
SIZES = [(1, 1), (3, 7), (1, 2048), (700, 64), (33, 1000), (129, 1001), (37, 4096), (6, 8192), (3, 8191), (2000, 264), (5000, 128),
         (9, 24), (257, 520), (65, 16), (31, 392)]


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from prefix_shared_chunkwise_gb300 import build
    build.build()


def _np(t):
    return None if t is None else t.double().cpu().numpy()


class Case:
    def __init__(self, C, D, dtype, form, seed=0, scale=0.4):
        post, act, res, pre = FORMS[form]
        td, self.r = DT[dtype]
        g = torch.Generator(device="cuda").manual_seed(seed + 31 * C + D)
        rand = lambda s=1.0: (s * torch.randn((C, D), generator=g, device="cuda")).to(td)
        w = lambda: 1 + 0.2 * torch.randn(D, generator=g, device="cuda")
        self.C, self.D, self.scale, self.act = C, D, scale, act or "linear"
        self.y, self.gate, self.res = rand(2.0), rand(2.0) if act else None, rand(3.0) if res else None
        self.post, self.pre = w() if post else None, w() if pre else None
        self.dn, self.dh = rand() if pre else None, rand() if res or not pre else None

    def kw(self):
        return dict(post_weight=self.post, gate=self.gate, gate_act=self.act, scale=self.scale, pre_weight=self.pre)

    def forward(self, **kw):
        return block_norm_fwd(self.y, residual=self.res, eps=EPS, **self.kw(), **kw)

    def backward(self, h, r1, r2, **kw):
        return block_norm_bwd(self.y, h, self.dn, self.dh, **self.kw(), rstd_post=r1, rstd_pre=r2, **kw)

    def check_forward(self):
        h, n, r1, r2 = self.forward()
        torch.cuda.synchronize()
        y, g, res = _np(self.y), _np(self.gate), _np(self.res)
        rh, rn, rr1, rr2 = ref.forward(y, _np(self.post), g, self.act, self.scale, res, _np(self.pre), EPS)
        k = (self.D / 64 + 12) * U
        z = 0.0 if g is None or self.act == "linear" else np.abs(g)
        block = np.abs(rh - (0.0 if res is None else res))
        e = (k + (16 + 1.5 * z) * U) * block + U * (np.abs(rh) + (0 if res is None else np.abs(res)))
        assert np.all(np.abs(_np(h) - rh) <= self.r * np.abs(rh) + e + 1e-37)
        if r1 is not None:
            assert np.all(np.abs(_np(r1) - rr1) <= k * rr1)
        if r2 is not None:
            k2 = k + np.sum(np.abs(rh) * e, axis=1) / (np.sum(rh * rh, axis=1) + self.D * EPS)
            assert np.all(np.abs(_np(r2) - rr2) <= k2 * rr2)
            bound = (self.r + k2[:, None] + 3 * U) * np.abs(rn) + np.abs(rr2[:, None] * _np(self.pre)) * e
            assert np.all(np.abs(_np(n) - rn) <= bound + 1e-37)
        assert (n is None) == (self.pre is None) and (r1 is None) == (self.post is None)
        return h, r1, r2

    def check_backward(self, h, r1, r2):
        got = self.backward(h, r1, r2)
        torch.cuda.synchronize()
        y, g, post, pre = _np(self.y), _np(self.gate), _np(self.post), _np(self.pre)
        n1, n2 = _np(r1), _np(r2)
        want = ref.backward(y, _np(h), _np(self.dn), _np(self.dh), post, g, self.act, self.scale, pre, n1, n2)
        rows = (self.D / 32 + 20) * U
        size = np.zeros_like(y) if self.dh is None else np.abs(_np(self.dh))
        if pre is not None:
            N, t = np.abs(_np(h) * n2[:, None]), np.abs(_np(self.dn) * pre)
            size = size + n2[:, None] * (t + N * np.mean(t * N, axis=1, keepdims=True))
            assert np.all(np.abs(_np(got["dpre_weight"]) - want["dpre_weight"]) <= (self.C + 20) * U * np.sum(np.abs(_np(self.dn)) * N, axis=0) + 1e-37)
        e_d = rows * size
        if got["dresidual"] is not None:
            assert np.all(np.abs(_np(got["dresidual"]) - want["dresidual"]) <= self.r * np.abs(want["dresidual"]) + e_d + 1e-37)
        Y = y if post is None else y * n1[:, None]
        value, z = 1.0, 0.0
        if g is not None:
            value, slope = ref.gate(g, self.act)
            z = 0.0 if self.act == "linear" else np.abs(g)
            q = 0.0 if self.act == "linear" else ref.gate(g, "sigmoid")[0]
            u = np.abs(self.scale * Y * (1 if post is None else post))
            bound = u * (np.abs(slope) * e_d + (np.abs(want["dresidual"]) + e_d) * (12 + 2 * z) * U * (q * (1 + z)))
            assert np.all(np.abs(_np(got["dgate"]) - want["dgate"]) <= (self.r + 8 * U) * np.abs(want["dgate"]) + bound + 1e-37)
        e = np.abs(want["d_block"])
        e_e = np.abs(self.scale * value) * e_d + (14 + 1.5 * z) * U * e
        bound = e_e
        if post is not None:
            Y, w = np.abs(Y), np.abs(post)
            mean = lambda v: v + Y * np.mean(v * Y, axis=1, keepdims=True)
            bound = n1[:, None] * (mean(w * e_e) + rows * mean(w * e))
            dw = np.abs(_np(got["dpost_weight"]) - want["dpost_weight"])
            assert np.all(dw <= (self.C + 20) * U * np.sum(e * Y, axis=0) + np.sum(e_e * Y, axis=0) + 1e-37)
        assert np.all(np.abs(_np(got["dy"]) - want["dy"]) <= self.r * np.abs(want["dy"]) + bound + 1e-37)
        again = self.backward(h, r1, r2)
        assert all(torch.equal(got[n], again[n]) for n in got if got[n] is not None)
        return got


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("form", sorted(FORMS))
@pytest.mark.parametrize("C,D", SIZES)
def test_forward_and_backward(C, D, form, dtype):
    c = Case(C, D, dtype, form)
    c.check_backward(*c.check_forward())


def test_many_short_rows():
    c = Case(70_001, 128, "bf16", "heads")
    c.check_backward(*c.check_forward())


@pytest.mark.parametrize("form", ["all", "pre", "post"])
@pytest.mark.parametrize("D", [2048, 100, 1003])
def test_in_place(form, D):
    c = Case(300, D, "bf16", form)
    h, n, r1, r2 = c.forward()
    d = c.backward(h, r1, r2)
    res = c.res.clone()
    h2, n2, _, _ = block_norm_fwd(c.y, residual=res, eps=EPS, **c.kw(), h=res, n=c.y.clone() if n is not None else None)
    assert h2 is res and torch.equal(h2, h) and (n is None or torch.equal(n2, n))
    y, dn, dh, gate = c.y.clone(), None if c.dn is None else c.dn.clone(), c.dh.clone(), None if c.gate is None else c.gate.clone()
    kw = dict(c.kw(), gate=gate)
    got = block_norm_bwd(y, h, dn, dh, **kw, rstd_post=r1, rstd_pre=r2, dy=y, dresidual=dh, dgate=gate)
    assert all(torch.equal(got[k], d[k]) for k in d if d[k] is not None)
    assert got["dy"] is y and got["dresidual"] is dh



# rows that begin inside a vector: up to its last value, over more rows than are resident, shorter than a
# vector, as wide as whole vectors of such rows may be, and one wider
RAGGED = [(1, 3), (11, 5), (50_003, 3), (5, 65), (40_001, 67), (20_000, 100), (9001, 250), (5000, 129), (3001, 513), (2501, 1025),
          (901, 2047), (400, 4095), (333, 4089), (40, 8185), (3, 8186), (6, 8189)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("form", ["all", "heads", "bare"])
@pytest.mark.parametrize("C,D", RAGGED)
def test_rows_that_are_not_whole_vectors(C, D, form, dtype):
    c = Case(C, D, dtype, form)
    c.check_backward(*c.check_forward())


@pytest.mark.parametrize("C,D", [(3000, 1003), (30_000, 61), (700, 4001)])
def test_neighbours_of_rows_that_begin_inside_a_vector(C, D):
    """Nothing of a row reaches the next, which shares its first or last 16 bytes; in place neither."""
    c = Case(C, D, "bf16", "all")
    h, n, r1, r2 = c.forward()
    d = c.backward(h, r1, r2)
    res, y = c.res.clone(), c.y.clone()
    got = block_norm_fwd(y, residual=res, eps=EPS, **c.kw(), h=res, n=y)
    assert got[0] is res and torch.equal(res, h) and torch.equal(y, n)
    rows = torch.arange(C, device="cuda")
    bad, good = rows % 3 == 1, rows % 3 != 1
    odd = torch.tensor([float("nan"), float("inf"), -float("inf")], device="cuda").bfloat16()
    for t in (c.y, c.gate, c.res, c.dn, c.dh):
        t[bad] = odd[torch.randint(0, 3, (D,), device="cuda")]
    h2, n2, s1, s2 = c.forward()
    h[bad] = float("nan")
    d2 = c.backward(h, r1, r2)
    assert torch.equal(h2[good], h[good]) and torch.equal(n2[good], n[good]) and torch.equal(s1[good], r1[good]) and torch.equal(s2[good], r2[good])
    for k in ("dy", "dresidual", "dgate"):
        assert torch.equal(d2[k][good], d[k][good])


def test_gate_far_out_and_rows_of_nothing():
    c = Case(4, 512, "fp32", "all")
    c.gate[0] = 90.0
    c.gate[1] = -90.0
    c.y[2] = 0
    c.res[2] = 0
    h, r1, r2 = c.check_forward()
    c.check_backward(h, r1, r2)
    assert bool((h[2] == 0).all())
    # what is not finite stays in its row
    base = c.forward()
    c.y[1, 5] = float("nan")
    got = c.forward()
    for a, b in zip(base, got):
        keep = [0, 2, 3]
        assert torch.equal(a[keep], b[keep])
    assert bool(got[1][1].isnan().all())


def test_captured_and_on_another_stream():
    c = Case(1000, 2048, "bf16", "all")
    h, n, r1, r2 = c.forward()
    want = [h, n, *c.backward(h, r1, r2).values()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a, b, q1, q2 = c.forward(stream=s)
    got = [a, b, *c.backward(a, q1, q2, stream=s).values()]
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, b, q1, q2 = c.forward()
        got = [a, b, *c.backward(a, q1, q2).values()]
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        assert all(torch.equal(x, y) for x, y in zip(want, got))


def test_no_rows():
    e = torch.empty((0, 64), device="cuda")
    w = torch.ones(64, device="cuda")
    h, n, r1, r2 = block_norm_fwd(e, post_weight=w, pre_weight=w)
    assert h.shape == n.shape == (0, 64) and r1.shape == (0,)
    d = block_norm_bwd(e, h, e, post_weight=w, pre_weight=w, rstd_post=r1, rstd_pre=r2)
    assert bool((d["dpost_weight"] == 0).all()) and bool((d["dpre_weight"] == 0).all())
