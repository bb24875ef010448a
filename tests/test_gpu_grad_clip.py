"""GPU parity of harts_grad_norm / harts_grad_clip against the fp64 oracle (oracle/tail.py).

Bounds.  u = 2^-24.  Squares are added in fp32 chains of at most 16 + 4 additions before fp64
takes over, so the sum is within 20 u and the norm within 10 u + u (its rounding).  A clipped
value carries the coefficient (11 u + u) and one product: within 14 u, plus half a step of its
own type (bf16 2^-8)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import tail
from prefix_shared_chunkwise_gb300.api import GradSet

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from prefix_shared_chunkwise_gb300 import build
    build.build()


def _grads(sizes, kinds, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, generator=g, device="cuda") * scale).to(kinds[i % len(kinds)]) for i, n in enumerate(sizes)]


def _check(grads, outs, max_norm):
    norm, ref = tail.grad_clip([g.double().cpu().numpy() for g in grads], max_norm)
    s = GradSet(grads, outs)
    only = s.norm()
    got = s.clip(max_norm)
    torch.cuda.synchronize()
    assert abs(float(only) - norm) <= 11 * U * norm
    assert float(only) == float(got)
    for o, r in zip(s.outs, ref):
        half = 2.0 ** -8 if o.dtype == BF else U
        assert np.all(np.abs(o.double().cpu().numpy() - r) <= (half + 14 * U) * np.abs(r) + 1e-38)


@pytest.mark.parametrize("kinds,out", [((F32,), F32), ((BF,), BF), ((BF,), F32), ((F32,), BF), ((BF, F32), None)])
@pytest.mark.parametrize("sizes", [(1,), (7, 1, 0, 33), (2048,), (100_003, 5, 64, 0, 4097), (3_000_001, 16)])
def test_norm_and_clip(sizes, kinds, out):
    grads = _grads(sizes, kinds, 1)
    outs = [torch.full_like(g, 9.0, dtype=g.dtype if out is None else out) for g in grads]
    total = sum(sizes) ** 0.5
    _check(grads, outs, 0.3 * total)
    _check(grads, outs, 10.0 * total)               # nothing to clip: a copy


def test_unaligned_views():
    """Gradients and outputs that start at every offset of a 16-byte line."""
    for kind in (BF, F32):
        for a in range(8):
            for b in (0, 1, 3):
                base = _grads([5000], [kind], a)[0]
                out = torch.zeros(5000, dtype=kind, device="cuda")
                _check([base[a:a + 4001]], [out[b:b + 4001]], 10.0)
                assert float(out[:b].abs().sum()) == 0 and float(out[b + 4001:].abs().sum()) == 0


def test_many_tensors():
    sizes = [(i * 37) % 611 for i in range(1300)]   # more than two launches' worth, empty ones among them
    grads = _grads(sizes, (BF, F32), 2)
    _check(grads, [torch.empty_like(g) for g in grads], 50.0)


def test_in_place():
    grads = _grads([1000, 77, 300_000], (F32, BF), 3)
    keep = [g.clone() for g in grads]
    s = GradSet(grads)
    n = float(s.clip(1e9))
    assert all(torch.equal(a, b) for a, b in zip(grads, keep))
    norm, ref = tail.grad_clip([g.double().cpu().numpy() for g in keep], 2.0)
    s.clip(2.0)
    for g, r in zip(grads, ref):
        half = 2.0 ** -8 if g.dtype == BF else U
        assert np.all(np.abs(g.double().cpu().numpy() - r) <= (half + 14 * U) * np.abs(r) + 1e-38)
    assert abs(n - norm) <= 11 * U * norm


def test_squares_beyond_fp32():
    g = [torch.full((5000,), 3e30, device="cuda"), torch.full((9,), 1.0, device="cuda", dtype=BF)]
    _check(g, [torch.empty_like(t) for t in g], 1e30)


def test_zero_and_empty():
    z = [torch.zeros(100, device="cuda"), torch.zeros(0, device="cuda")]
    out = [torch.ones_like(t) for t in z]
    assert float(GradSet(z, out).clip(0.0)) == 0 and float(out[0].abs().sum()) == 0
    assert float(GradSet([]).norm()) == 0 and float(GradSet([]).clip(1.0)) == 0


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_not_finite(bad):
    grads = _grads([3000, 50], (F32, BF), 4)
    grads[1][7] = bad
    outs = [torch.empty_like(g) for g in grads]
    n = GradSet(grads, outs).clip(0.1)
    torch.cuda.synchronize()
    assert not torch.isfinite(n)
    assert all(torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float())) for a, b in zip(grads, outs))


def test_graph_and_stream():
    grads = _grads([10_000, 333], (BF, F32), 5)
    outs = [torch.empty_like(g) for g in grads]
    s = GradSet(grads, outs)
    n = torch.empty((), device="cuda")
    s.clip(1.0, norm=n)
    want, wn = [o.clone() for o in outs], float(n)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.clip(1.0, norm=n)
    for o in outs:
        o.zero_()
    n.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want)) and float(n) == wn


@pytest.mark.parametrize("kind", [BF, F32])
@pytest.mark.parametrize("scale", [1e-19, 1e-20, 1e-25, 1e-35])
def test_squares_below_fp32(kind, scale):
    """Values whose squares fp32 holds as zero or with few bits.  The norm's own bound; a clipped
    value's is its relative one, with half of the type's smallest step (2^-134 bf16, 2^-150 fp32)
    where it is not normal."""
    for sizes in ((1,), (5001, 3, 700_001), (100, 0, 40)):
        grads = _grads(sizes, [kind], 6, scale)
        if sizes[0] == 100:                         # among zeros, and one tensor of them
            grads[0][1:] = 0
            grads[2].zero_()
        outs = [torch.empty_like(g) for g in grads]
        full = float(np.sqrt(sum(float(g.double().square().sum()) for g in grads)))
        norm, ref = tail.grad_clip([g.double().cpu().numpy() for g in grads], 0.25 * full)
        s = GradSet(grads, outs)
        got = s.clip(0.25 * full)
        assert abs(float(s.norm()) - norm) <= 11 * U * norm and abs(float(got) - norm) <= 11 * U * norm
        half, low = (2.0 ** -8, 2.0 ** -134) if kind == BF else (U, 2.0 ** -150)
        for o, r in zip(outs, ref):
            assert np.all(np.abs(o.double().cpu().numpy() - r) <= (half + 14 * U) * np.abs(r) + low)


def test_small_values_next_to_large_ones():
    """A block of tiny values beside one whose squares are ordinary: the norm is the latter's."""
    grads = [*_grads([300_000], [F32], 7, 1e-30), *_grads([300_000], [BF], 8)]
    _check(grads, [torch.empty_like(g) for g in grads], 1.0)



def test_norm_beyond_fp32():
    """Finite values whose norm fp32 does not hold: *norm is infinite, and the gradients pass
    unscaled, as with every norm that is not finite."""
    grads = [torch.full((5000,), 3e38, device="cuda"), torch.ones(9, device="cuda", dtype=BF)]
    outs = [torch.zeros_like(g) for g in grads]
    n = GradSet(grads, outs).clip(1.0)
    torch.cuda.synchronize()
    assert torch.isinf(n) and all(torch.equal(o, g) for o, g in zip(outs, grads))


@pytest.mark.parametrize("kind,out", [(F32, F32), (BF, BF), (F32, BF), (BF, F32)])
def test_coefficients_below_fp32(kind, out):
    """max_norm / norm that fp32 holds with few bits or as zero, from 2^-120 to 2^-150."""
    for max_norm, value in ((1e-5, 1e31), (1e-8, 1e31), (1e-12, 3e30), (3e-14, 3e30)):
        grads = [torch.full((5003,), value, device="cuda", dtype=kind), torch.full((9,), -value, device="cuda", dtype=kind)]
        _check(grads, [torch.zeros_like(g, dtype=out) for g in grads], max_norm)
    zero = torch.ones(9, device="cuda", dtype=out)
    GradSet([torch.full((9,), 1.0, device="cuda", dtype=kind)], [zero]).clip(0.0)
    assert float(zero.abs().sum()) == 0
