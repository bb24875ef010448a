"""GPU parity of harts_linear_logprob_fwd / _bwd against the fp64 oracle (oracle/tail.py) on
the same bf16 inputs.

Bounds.  u = 2^-23 bounds an fp32 addition on the tensor cores (which may truncate).  A logit
sums D products: off by e_z = D u |scale| max_v sum_i |x_i w_i|.  lse is off by at most that,
plus the joined exponentials (8 u) and its rounding (u |lse|); logp by that plus its own dot
product.  dz = -G p + g carries e_z + e_lse + 8 u in p, and one rounding to bf16 (half a step:
2^-8); dx adds V terms, dweight C terms: elementwise
  |d - ref| <= ((2^-8 + 8 u) |dz| + (e_z + e_lse) |G| p) |w| + n u |dz| |w| + 2^-8 |ref|,
with the sums over |.| formed here in fp64."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import tail
from prefix_shared_chunkwise_gb300.api import Plan, linear_logprob_bwd, linear_logprob_fwd, semantic_map
from prefix_shared_chunkwise_gb300.synth import make_tree
from tests._parity import rel_l2

pytestmark = pytest.mark.gpu

U = 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from prefix_shared_chunkwise_gb300 import build
    build.build()


def _csr(sem_row, C):
    row_ptr = np.zeros(C + 1, np.int32)
    np.add.at(row_ptr, sem_row + 1, 1)
    return np.cumsum(row_ptr).astype(np.int32), np.argsort(sem_row, kind="stable").astype(np.int32)


def _case(C, V, D, S, seed, spread=2.0, labels=None):
    """Rows without positions, labels shared and distinct within a row, and positions without
    a label (-1 and V) all occur once S is large enough."""
    rng = np.random.default_rng(seed)
    bf = lambda a: torch.as_tensor(a, dtype=torch.float32).to(torch.bfloat16)
    x, w = bf(rng.standard_normal((C, D))), bf(rng.standard_normal((V, D)) * spread / D ** 0.5)
    sem_row = rng.integers(0, max(1, C - C // 5), size=S)
    target = rng.integers(0, V if labels is None else min(V, labels), size=S)
    target[rng.random(S) < 0.05] = -1
    target[rng.random(S) < 0.02] = V
    g = rng.standard_normal(S).astype(np.float32)
    g[rng.random(S) < 0.1] = 0
    return x, w, sem_row.astype(np.int64), target.astype(np.int64), g


def _dev(a):
    return torch.as_tensor(a, device="cuda")


def _run_fwd(x, w, sem_row, target, scale, **kw):
    row_ptr, row_sem = _csr(sem_row, x.shape[0])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    logp, lse = linear_logprob_fwd(x.cuda(), w.cuda(), _dev(row_ptr), _dev(row_sem), _dev(target.astype(np.int32)),
                                   scale=scale, error=err, **kw)
    torch.cuda.synchronize()
    assert int(err) == 0
    return logp, lse


def _errors(x, w, scale, lse):
    xa, wa = np.abs(x.double().numpy()), np.abs(w.double().numpy())
    ez = x.shape[1] * U * abs(scale) * (xa @ wa.T).max(axis=1)
    return ez, ez + 8 * U + U * np.abs(lse)


SIZES = [(1, 1, 8, 1), (1, 5, 8, 3), (3, 64, 64, 10), (1, 40_001, 256, 1), (5, 257, 72, 40), (127, 255, 128, 300),
         (128, 256, 64, 0), (129, 1000, 200, 700), (300, 2049, 1032, 900), (777, 4099, 136, 1000)]


@pytest.mark.parametrize("C,V,D,S", SIZES)
@pytest.mark.parametrize("scale", [1.0, 0.6])
def test_forward(C, V, D, S, scale):
    x, w, sem_row, target, _ = _case(C, V, D, S, 1)
    logp, lse = _run_fwd(x, w, sem_row, target, scale)
    rl, re = tail.linear_logprob_fwd(x.double().numpy(), w.double().numpy(), sem_row, target, scale)
    ez, el = _errors(x, w, scale, re)
    assert np.all(np.abs(lse.cpu().numpy() - re) <= el)
    assert np.all(np.abs(logp.cpu().numpy() - rl) <= (ez + el)[sem_row] + U * np.abs(rl)) if S else True


def _check_bwd(x, w, sem_row, target, g, scale, piece=0):
    C, V, D = x.shape[0], w.shape[0], x.shape[1]
    x64, w64 = x.double().numpy(), w.double().numpy()
    _, re = tail.linear_logprob_fwd(x64, w64, sem_row, target, scale)
    row_ptr, row_sem = _csr(sem_row, C)
    args = (x.cuda(), w.cuda(), _dev(row_ptr), _dev(row_sem), _dev(target.astype(np.int32)),
            _dev(re.astype(np.float32)), _dev(g))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(scale=scale, piece=piece, error=err)
    dx, dw = linear_logprob_bwd(*args, **kw, dx=torch.full_like(args[0], 7), dweight=torch.full_like(args[1], 7))
    dx2, dw2 = linear_logprob_bwd(*args, **kw)
    torch.cuda.synchronize()
    assert int(err) == 0
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)       # no order of additions left open
    rdx, rdw = tail.linear_logprob_bwd(x64, w64, sem_row, target, g, scale)
    ez, el = _errors(x, w, scale, re)
    keep = (target >= 0) & (target < V)
    G, Ga = np.zeros(C), np.zeros(C)
    np.add.at(G, sem_row[keep], g[keep].astype(np.float64))
    np.add.at(Ga, sem_row[keep], np.abs(g[keep]).astype(np.float64))
    p = np.exp(scale * (x64 @ w64.T) - re[:, None])
    own = np.zeros((C, V))
    np.add.at(own, (sem_row[keep], target[keep]), np.abs(g[keep]).astype(np.float64))
    dz = np.abs(G)[:, None] * p + own                          # |dz| at most
    off = (2.0 ** -8 + 8 * U) * dz + (ez + el)[:, None] * np.abs(G)[:, None] * p + len(g) * U * (Ga[:, None] * p + own)
    for got, ref, o, n in ((dx, rdx, abs(scale) * (off @ np.abs(w64)), V), (dw, rdw, abs(scale) * (off.T @ np.abs(x64)), C)):
        size = abs(scale) * ((dz @ np.abs(w64)) if n == V else (dz.T @ np.abs(x64)))
        got = got.double().cpu().numpy()
        assert np.all(np.abs(got - ref) <= o + n * U * size + 2.0 ** -8 * np.abs(ref) + 1e-37)
        if np.linalg.norm(ref) > 0:
            assert rel_l2(got, ref) <= 1e-2
    empty = np.setdiff1d(np.arange(C), sem_row[keep])
    assert np.all(dx.float().cpu().numpy()[empty] == 0)


@pytest.mark.parametrize("C,V,D,S", SIZES)
@pytest.mark.parametrize("scale", [1.0, 0.6])
def test_backward(C, V, D, S, scale):
    _check_bwd(*_case(C, V, D, S, 2), scale)


@pytest.mark.parametrize("piece", [1, 256, 700, 2048, 100_000])
def test_backward_in_pieces(piece):
    _check_bwd(*_case(150, 2049, 136, 400, 3), 0.8, piece)


def test_many_positions_on_one_row():
    """All positions on few rows, with few labels and with many."""
    for labels in (3, None):
        x, w, _, target, g = _case(4, 999, 64, 500, 4, labels=labels)
        sem_row = np.where(np.arange(500) < 450, 2, 0).astype(np.int64)
        _check_bwd(x, w, sem_row, target, g, 1.0)
        logp, lse = _run_fwd(x, w, sem_row, target, 1.0)
        rl, re = tail.linear_logprob_fwd(x.double().numpy(), w.double().numpy(), sem_row, target)
        ez, el = _errors(x, w, 1.0, re)
        assert np.all(np.abs(logp.cpu().numpy() - rl) <= (ez + el)[sem_row] + U * np.abs(rl))


@pytest.mark.parametrize("labels", [1, 40, None])
def test_thousands_of_positions_on_one_row(labels):
    """3,000 positions of one row with one label, with 40 and with hundreds of distinct ones:
    shared labels add up, distinct ones are found by the tiles they lie in."""
    rng = np.random.default_rng(9)
    x, w, _, _, _ = _case(3, 5003, 64, 1, 9)
    S = 3100
    sem_row = np.where(np.arange(S) < 3000, 1, 2).astype(np.int64)
    target = rng.integers(0, 5003 if labels is None else labels, size=S)
    target[::50] = -1
    g = rng.standard_normal(S).astype(np.float32)
    _check_bwd(x, w, sem_row, target, g, 1.0)


def test_gradients_that_cancel():
    """Positions of one label whose gradients cancel, and rows whose G is zero."""
    x, w, _, _, _ = _case(4, 300, 64, 1, 10)
    sem_row = np.array([0, 0, 1, 1, 2, 2, 2], np.int64)
    target = np.array([5, 5, 7, 9, 250, 3, 3], np.int64)
    g = np.array([1.5, -1.5, 2.0, -2.0, 1.0, 0.5, -0.5], np.float32)
    _check_bwd(x, w, sem_row, target, g, 1.0)


def test_peaked_rows():
    """Logits of spread 60: softmax rows close to one-hot, exponentials that underflow."""
    x, w, sem_row, target, g = _case(40, 700, 128, 100, 5, spread=60.0)
    logp, lse = _run_fwd(x, w, sem_row, target, 1.0)
    rl, re = tail.linear_logprob_fwd(x.double().numpy(), w.double().numpy(), sem_row, target)
    ez, el = _errors(x, w, 1.0, re)
    assert np.all(np.abs(lse.cpu().numpy() - re) <= el)
    assert np.all(np.abs(logp.cpu().numpy() - rl) <= (ez + el)[sem_row] + U * np.abs(rl))
    _check_bwd(x, w, sem_row, target, g, 1.0)


def test_gradient_against_differences():
    """<dx, d> and <dweight, d> against central differences of the forward kernel's
    sum_s g_s logp[s].  Inputs on a grid of 2^-3 below 4 and steps of 2^-5 are exact in bf16;
    the third-order term is ~ (step |w|)^2 < 1e-3 of the value, bf16 rounding of the gradient
    2^-8 of its terms: 2 % of the sum of absolute terms over sqrt(n) is far above both."""
    rng = np.random.default_rng(6)
    C, V, D, S, step = 20, 300, 64, 60, 2.0 ** -5
    grid = lambda a: torch.as_tensor(np.clip(np.round(a * 8) / 8, -3.5, 3.5), dtype=torch.float32)
    x, w = grid(rng.standard_normal((C, D))), grid(rng.standard_normal((V, D)) * 0.3)
    sem_row, target = rng.integers(0, C, S), rng.integers(0, V, S)
    g = rng.standard_normal(S).astype(np.float32)
    row_ptr, row_sem = _csr(sem_row, C)
    idx = (_dev(row_ptr), _dev(row_sem), _dev(target.astype(np.int32)))
    scale = 0.25

    def loss(a, b):
        logp, lse = linear_logprob_fwd(a.to(torch.bfloat16).cuda(), b.to(torch.bfloat16).cuda(), *idx, scale=scale)
        return float((logp.double() * _dev(g).double()).sum()), lse

    _, lse = loss(x, w)
    dx, dw = linear_logprob_bwd(x.to(torch.bfloat16).cuda(), w.to(torch.bfloat16).cuda(), *idx, lse, _dev(g), scale=scale)
    for grad, base, put in ((dx, x, lambda a: (a, w)), (dw, w, lambda a: (x, a))):
        d = torch.as_tensor(rng.choice([-1.0, 1.0], size=tuple(base.shape)), dtype=torch.float32)
        num = (loss(*put(base + step * d))[0] - loss(*put(base - step * d))[0]) / (2 * step)
        terms = grad.double().cpu() * d.double()
        assert abs(float(terms.sum()) - num) <= 0.02 * float(terms.square().sum().sqrt()) * 3


def test_semantic_map_of_a_forest():
    """A forest's own semantic map at an odd vocabulary: shared rows carry several positions."""
    parent, seg_len = make_tree("fig1_fp32")
    pl = Plan(parent, seg_len, 64)
    sem_row, row_ptr, row_sem = semantic_map(pl)
    C, S, V, D = pl.info["C"], len(sem_row), 5003, 256
    x, w, _, target, g = _case(C, V, D, S, 7)
    _check_bwd(x, w, sem_row.astype(np.int64), target, g, 1.0)


def test_large_row_offsets():
    """A weight whose rows pass 2^31 elements: the last vocabulary entries decide the result."""
    V, D, C = 600_000, 4096, 3
    w = torch.zeros((V, D), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    w[-300:] = torch.randn((300, D), generator=g, device="cuda").to(torch.bfloat16)
    x = torch.randn((C, D), generator=g, device="cuda").to(torch.bfloat16)
    ptr = torch.arange(C + 1, dtype=torch.int32, device="cuda")
    tgt = torch.tensor([V - 1, V - 299, 5], dtype=torch.int32, device="cuda")
    logp, lse = linear_logprob_fwd(x, w, ptr, ptr[:C].clone(), tgt)
    z = x.double() @ w[-300:].double().t()
    re = torch.logsumexp(torch.cat([z, torch.zeros((C, 1), dtype=torch.float64, device="cuda") + np.log(V - 300)], 1), 1)
    rl = torch.stack([z[0, 299], z[1, 1], 0 * z[2, 0]]) - re
    size = float((x.double().abs() @ w[-300:].double().abs().t()).max())
    tol = 2 * D * U * size + 20 * U + 4 * U * float(re.abs().max())
    assert float((lse.double() - re).abs().max()) <= tol and float((logp.double() - rl).abs().max()) <= tol
    dx, dw = linear_logprob_bwd(x, w, ptr, ptr[:C].clone(), tgt, lse, torch.ones(C, device="cuda"))
    p = torch.exp(z - re[:, None])
    dz = -p
    dz[0, 299] += 1
    dz[1, 1] += 1
    assert rel_l2(dw[-300:].double().cpu().numpy(), (dz.t() @ x.double()).cpu().numpy()) <= 1e-2
    assert rel_l2(dx.double().cpu().numpy(), (dz @ w[-300:].double()).cpu().numpy()) <= 1e-2


def test_no_rows_and_stream_and_graph():
    x, w, sem_row, target, g = _case(70, 500, 64, 90, 8)
    row_ptr, row_sem = _csr(sem_row, 70)
    a = (x.cuda(), w.cuda(), _dev(row_ptr), _dev(row_sem), _dev(target.astype(np.int32)))
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    z1 = torch.zeros(1, dtype=torch.int32, device="cuda")
    logp, lse = linear_logprob_fwd(e, a[1], z1, none, none)
    dx, dw = linear_logprob_bwd(e, a[1], z1, none, none, lse, logp)
    assert logp.numel() == 0 and float(dw.float().abs().sum()) == 0
    logp, lse = linear_logprob_fwd(*a)
    dx, dw = linear_logprob_bwd(*a, lse, _dev(g))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    l2, e2 = linear_logprob_fwd(*a, stream=st)
    st.synchronize()
    assert torch.equal(l2, logp) and torch.equal(e2, lse)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    dx3, dw3, dl = torch.zeros_like(dx), torch.zeros_like(dw), _dev(g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        linear_logprob_bwd(*a, lse, dl, dx=dx3, dweight=dw3, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(dx3, dx) and torch.equal(dw3, dw)


@pytest.mark.parametrize("C,V,D,scale", [(1, 5003, 2048, 1.0), (6, 321, 1032, 1.0), (130, 2050, 512, -0.5), (300, 777, 2048, 1.0)])
def test_an_entry_with_nearly_all_the_probability(C, V, D, scale):
    """Rows that lean on one entry v* (the last, one in either half of a tile, any), labelled with
    it and with another.  Its logit is formed in fp32: with Z = sum |x_i w_i| an error of at most
    e = (16 D / 1024 + 12) u Z (sixteen products in a row for each 1024, then sums over threads,
    and the scaling).  The other entries' probabilities, q in all, are off by e_z of the module's
    bound.  At most 40 additions go onto a sum that holds the largest term (16 in its 32 columns,
    8 across the tile's halves, 16 across tiles and threads; u / 2 each), and exponentials take
    4 u.  So lse is off by e + q (e + e_z) + 24 u + u |lse|, and the log-probability of v* by
    q (e + e_z) + 24 u; without the fp32 product it would be off by what the tensor cores
    truncate, some 1e-6 of the logit whatever q is.  The other label's logit is an fp32 product
    too."""
    rng = np.random.default_rng(C + V)
    bf = lambda a: torch.as_tensor(a, dtype=torch.float32).to(torch.bfloat16)
    w = bf(rng.standard_normal((V, D)) * 2 / D ** 0.5)
    main = rng.integers(0, V, size=C)
    main[:4] = [V - 1, 0, 37, 250][:C]
    x = bf(rng.standard_normal((C, D)) + 5 / scale * w.double().numpy()[main])
    sem_row = np.concatenate([np.arange(C), np.arange(C)])
    target = np.concatenate([main, (main + 1 + rng.integers(0, V - 1, size=C)) % V])
    logp, lse = (a.double().cpu().numpy() for a in _run_fwd(x, w, sem_row, target, scale))
    ref_logp, ref_lse = tail.linear_logprob_fwd(x.double().numpy(), w.double().numpy(), sem_row, target, scale)
    xa, wa = np.abs(x.double().numpy()), np.abs(w.double().numpy())
    fp32 = lambda v: (D / 1024 * 16 + 12) * U * abs(scale) * (xa * wa[v]).sum(axis=1)
    e, (ez, _) = fp32(main), _errors(x, w, scale, ref_lse)
    q = -np.expm1(ref_logp[:C])
    assert (np.abs(lse - ref_lse) <= e + q * (e + ez) + 24 * U + U * np.abs(ref_lse)).all()
    assert (np.abs(logp - ref_logp)[:C] <= q * (e + ez) + 24 * U).all()
    assert (np.abs(logp - ref_logp)[C:] <= fp32(target[C:]) + e + q * (e + ez) + 24 * U + U * np.abs(ref_logp[C:])).all()
    assert np.median(q) < 0.05


@pytest.mark.parametrize("C,V,D,S", [(192, 515, 72, 300), (193, 770, 200, 300), (256, 900, 1032, 400), (257, 513, 136, 400)])
@pytest.mark.parametrize("scale", [1.0, -0.7])
def test_rows_around_the_cuts(C, V, D, S, scale):
    """Row counts on either side of where blocks pair up and where X is copied first; a negative
    scale turns the largest logit into the smallest accumulator."""
    test_forward(C, V, D, S, scale)
    _check_bwd(*_case(C, V, D, S, 6), scale)


@pytest.mark.parametrize("scale", [0.0, -1.0, 1.0])
def test_equal_logits(scale):
    """Entries that are all equal, and that differ in one: every one is the largest."""
    C, V, D = 130, 300, 64
    x = torch.ones(C, D, dtype=torch.bfloat16)
    w = torch.full((V, D), 0.125, dtype=torch.bfloat16)
    w[V - 1] = 0.25
    sem_row, target = np.arange(C), np.arange(C) * 2
    target[-1] = V - 1
    logp, lse = _run_fwd(x, w, sem_row, target, scale)
    rl, re = tail.linear_logprob_fwd(x.double().numpy(), w.double().numpy(), sem_row, target, scale)
    ez, el = _errors(x, w, scale, re)
    assert np.all(np.abs(lse.cpu().numpy() - re) <= el)
    assert np.all(np.abs(logp.cpu().numpy() - rl) <= ez + el + U * np.abs(rl))


@pytest.mark.parametrize("C,V,D", [(1, 5, 8), (3, 700, 64), (130, 1003, 136), (300, 2050, 72)])
@pytest.mark.parametrize("scale", [1.0, -0.5])
def test_not_finite_values_stay_visible(C, V, D, scale):
    """A NaN or an infinity in one vocabulary row reaches every row's softmax (an infinity as an
    infinite or undefined one), a NaN in one hidden row only that row's: lse and the positions'
    log-probabilities are then not finite, and those of the other rows as without it."""
    x, w, _, _, _ = _case(C, V, D, 1, 12)
    sem_row, target = np.arange(C), (np.arange(C) * 7) % V
    logp, lse = _run_fwd(x, w, sem_row, target, scale)
    assert torch.isfinite(lse).all() and torch.isfinite(logp).all()
    for v in {0, V // 2, V - 1}:
        for bad in (float("nan"), float("inf")):
            b = w.clone()
            b[v, D // 2] = bad
            got_logp, got_lse = _run_fwd(x, b, sem_row, target, scale)
            if np.isnan(bad):
                assert torch.isnan(got_lse).all() and torch.isnan(got_logp).all(), v
            else:                                   # z = -infinity leaves the entry out of the sum
                z = scale * (x.double() @ b.double().t())
                ref = torch.logsumexp(z, 1)
                seen = torch.isfinite(ref)
                assert not torch.isfinite(got_lse.cpu()[~seen]).any(), v
                assert torch.isfinite(got_lse.cpu()[seen]).all(), v
    b = x.clone()
    b[C // 2, 3] = float("nan")
    got_logp, got_lse = _run_fwd(b, w, sem_row, target, scale)
    rest = np.arange(C) != C // 2
    assert torch.isnan(got_lse[C // 2]) and torch.isnan(got_logp[C // 2])
    assert torch.equal(got_lse[rest], lse[rest]) and torch.equal(got_logp[rest], logp[rest])


@pytest.mark.parametrize("C,V,D", [(20, 2050, 72), (150, 2050, 136), (300, 1003, 72)])
def test_a_workspace_taken_again_for_other_labels(C, V, D):
    """Calls one after another in one workspace, each with its own labels and gradients: the bits
    of calls with a workspace of their own."""
    row_ptr, row_sem = (_dev(a) for a in _csr(np.arange(3 * C) % C, C))
    x, w, _, _, _ = _case(C, V, D, 1, 13)
    x, w = x.cuda(), w.cuda()
    rng = np.random.default_rng(13)
    sets = [(_dev(rng.integers(0, V, 3 * C).astype(np.int32)), _dev(rng.standard_normal(3 * C).astype(np.float32)))
            for _ in range(6)]
    lse = linear_logprob_fwd(x, w, row_ptr, row_sem, sets[0][0])[1]
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    shared = [linear_logprob_bwd(x, w, row_ptr, row_sem, t, lse, g, workspace=ws) for t, g in sets]
    for (t, g), got in zip(sets, shared):
        want = linear_logprob_bwd(x, w, row_ptr, row_sem, t, lse, g, workspace=torch.zeros_like(ws))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("V", [250, 40_003, 70_001])
def test_rows_with_many_distinct_labels(V):
    """Rows on either side of what one warp gathers (16 distinct labels), and one with thousands,
    each of them once, twice or more; labels of one, two and three bytes.  Gradients of a label that
    cancel, and positions without a label, among them."""
    rng = np.random.default_rng(V)
    D, sem_row, target = 64, [], []
    for row, (n, labels) in enumerate([(128, 16), (17, 17), (20_000, min(V, 12_000)), (0, 1), (700, 200)]):
        pool = rng.permutation(V)[:min(V, labels)]
        y = np.concatenate([pool, rng.choice(pool, max(0, n - len(pool)))])[:max(n, 0)]
        y = rng.permutation(y)
        if row == 4:
            y[::9] = [-1, V][0]
        sem_row.append(np.full(len(y), row))
        target.append(y)
    sem_row, target = np.concatenate(sem_row).astype(np.int64), np.concatenate(target).astype(np.int64)
    order = rng.permutation(len(sem_row))
    sem_row, target = sem_row[order], target[order]
    g = rng.standard_normal(len(sem_row)).astype(np.float32)
    twice = np.flatnonzero((sem_row == 2) & (target == target[sem_row == 2][0]))
    if len(twice) > 1:
        g[twice] = 0
        g[twice[0]], g[twice[1]] = 1.25, -1.25
    x, w, _, _, _ = _case(5, V, D, 1, 14)
    _check_bwd(x, w, sem_row, target, g, 1.0)


def test_distinct_labels_of_one_row_cost_what_they_are():
    """Eight times the distinct labels on one row take about eight times as long (plus what both
    calls share), not sixty-four; and the limit of the waits is for other things."""
    V, D = 157_184, 64
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((2, D), generator=gen, device="cuda").to(torch.bfloat16)
    w = (torch.randn((V, D), generator=gen, device="cuda") * 0.2).to(torch.bfloat16)
    lse = torch.logsumexp(x.double() @ w.double().t(), 1).float()

    def run(n):
        ptr = torch.tensor([0, n, n + 1], dtype=torch.int32, device="cuda")
        sem = torch.arange(n + 1, dtype=torch.int32, device="cuda")
        target = torch.randperm(V, generator=gen, device="cuda")[:n + 1].to(torch.int32)
        g = torch.randn(n + 1, generator=gen, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        best = float("inf")
        for _ in range(3):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            torch.cuda.synchronize()
            a.record()
            dx, dw = linear_logprob_bwd(x, w, ptr, sem, target, lse, g, error=err)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        assert int(err) == 0
        dz = -torch.exp(x.double() @ w.double().t() - lse.double()[:, None])
        dz *= torch.stack([g[:n].double().sum(), g[n].double()])[:, None]
        dz[0].index_add_(0, target[:n].long(), g[:n].double())
        dz[1, target[n].long()] += g[n].double()
        for got, ref in ((dx, dz @ w.double()), (dw, dz.t() @ x.double())):
            assert rel_l2(got.double().cpu().numpy(), ref.cpu().numpy()) <= 2.0 ** -7
        return best

    small, large = run(16_384), run(131_072)
    assert large <= 16 * small, (small, large)


def _bounds_of_the_forward(x, w, scale, lse, logp):
    """What errors the forward's rounding makes in relative L2, for sums of products of either sign.
    The tensor cores cut a running sum at every 16 products.  On average that takes 0.20 - 0.29 of
    2^-24 of a logit each time, of which the factor on the logits gives 0.25 back; what is left is
    0.05 D / 16, and a spread that grows with the root of their number.  lse is a mean of logits, to
    which exponentials and sums add some 8 roundings; a position's own logit is an fp32 sum in chains
    of D / 64, whose roundings mostly cancel."""
    D, u = x.shape[1], 2.0 ** -24
    z = np.abs(scale * (x.double().numpy() @ w.double().numpy().T)).max()
    rms = lambda a: np.sqrt(np.mean(np.square(a)))
    e = (0.05 * D / 16 + (D / 16) ** 0.5) * u * z + 8 * u
    own = ((D / 64) ** 0.5 + 8) * u * z
    return e / rms(lse) + 2 * u, (e + own) / max(rms(logp), 1e-30) + 2 * u


@pytest.mark.parametrize("C,V,D,S", [(1, 40_001, 256, 3), (20, 5003, 1032, 60), (129, 1000, 200, 700), (300, 2049, 1032, 900),
                                     (777, 4099, 136, 1000), (140, 3001, 2048, 300)])
@pytest.mark.parametrize("scale", [1.0, -0.625])
def test_forward_in_relative_l2(C, V, D, S, scale):
    """Beside the bound on each element, which adds up what could go wrong, one on all of them."""
    x, w, sem_row, target, _ = _case(C, V, D, S, 15)
    logp, lse = _run_fwd(x, w, sem_row, target, scale)
    rl, re = tail.linear_logprob_fwd(x.double().numpy(), w.double().numpy(), sem_row, target, scale)
    el, ep = _bounds_of_the_forward(x, w, scale, re, rl)
    assert rel_l2(lse.double().cpu().numpy(), re) <= el
    assert rel_l2(logp.double().cpu().numpy(), rl) <= ep


def _check_lse(x, w, scale, per_step):
    """lse where every logit is off by at most `per_step` 2^-24 of the largest for each 16 channels,
    and by the roundings of exponentials and sums."""
    C, V, D = x.shape[0], w.shape[0], x.shape[1]
    sem_row, target = np.arange(C), (np.arange(C) * 11) % V
    logp, lse = _run_fwd(x, w, sem_row, target, scale)
    x64, w64 = x.double().numpy(), w.double().numpy()
    rl, re = tail.linear_logprob_fwd(x64, w64, sem_row, target, scale)
    z = np.abs(scale * (x64 @ w64.T)).max(axis=1)
    el = per_step * D / 16 * 2.0 ** -24 * z + 24 * U + U * np.abs(re)
    assert np.all(np.abs(lse.cpu().numpy() - re) <= el)
    own = (D / 1024 * 16 + 12) * U * abs(scale) * np.array([np.abs(x64[c]) @ np.abs(w64[target[c]]) for c in range(C)])
    assert np.all(np.abs(logp.cpu().numpy() - rl) <= el + own + U * np.abs(rl))


@pytest.mark.parametrize("D", [256, 4096, 16_384])
def test_logits_that_are_exact(D):
    """Rows with one channel, and values on a coarse grid: the tensor cores cut nothing, and the
    factor of 1/4 2^-24 for each 16 channels that expects them to is all there is."""
    gen = torch.Generator().manual_seed(D)
    w = (torch.randn(300, D, generator=gen) * 4).bfloat16()
    x = torch.zeros(140, D)
    x[torch.arange(140), torch.randint(0, D, (140,), generator=gen)] = 1
    _check_lse(x.bfloat16(), w, 1.0, 0.25)
    grid = lambda *s: torch.randint(-2, 3, s, generator=gen).float()
    _check_lse(grid(20, D).bfloat16(), grid(300, D).bfloat16(), 4 / D ** 0.5, 0.25)


@pytest.mark.parametrize("D", [256, 4096, 16_384])
def test_logits_whose_products_have_one_sign(D):
    """Running sums that only grow are cut by less than two units of 2^-24 of the last one at every
    16 channels, less the quarter of one that the factor gives back (which is never more than was
    taken, but for logits that are exact)."""
    gen = torch.Generator().manual_seed(D)
    x, w = torch.rand(140, D, generator=gen).bfloat16(), torch.rand(300, D, generator=gen).bfloat16()
    for scale in (32 / D, -32 / D):
        _check_lse(x, w, scale, 2.0)


@pytest.mark.parametrize("C,V,D,S", [(20, 2049, 136, 60), (32, 1500, 72, 100), (193, 2049, 136, 500), (300, 1793, 72, 700),
                                     (520, 2500, 200, 900)])
@pytest.mark.parametrize("piece", [256, 1024])
def test_backward_in_pieces_of_other_forms(C, V, D, S, piece):
    """Several pieces with dZ in two terms (up to 32 rows) and on pairs of blocks (from 193)."""
    _check_bwd(*_case(C, V, D, S, 16), 0.8, piece)


@pytest.mark.parametrize("C,V,D", [(300, 700, 8), (257, 515, 40), (300, 2050, 56), (140, 300, 16), (20, 300, 24)])
def test_narrow_rows(C, V, D):
    """Rows narrower than one panel of 64 channels, on blocks alone and on pairs."""
    case = _case(C, V, D, 2 * C, 17)
    x, w, sem_row, target, _ = case
    logp, lse = _run_fwd(x, w, sem_row, target, 1.0)
    rl, re = tail.linear_logprob_fwd(x.double().numpy(), w.double().numpy(), sem_row, target)
    ez, el = _errors(x, w, 1.0, re)
    assert np.all(np.abs(lse.cpu().numpy() - re) <= el)
    assert np.all(np.abs(logp.cpu().numpy() - rl) <= (ez + el)[sem_row] + U * np.abs(rl))
    _check_bwd(*case, 1.0)
    _check_bwd(*case, 1.0, 256)


@pytest.mark.parametrize("C", [1, 31, 32])
def test_gradients_of_few_rows_are_rounded_once(C):
    """Rows whose label's dz lies halfway between two bf16 values, the entry that makes nearly all of
    the gradient.  In two terms dz is off by 2^-17, so that every element is the exact one rounded
    once: within half a step of bf16, 2^(floor(log2 |ref|) - 8), and what comes before it.  That is
    the sums (cut once for 16 products, and joined in at most 40 additions), and the softmax terms,
    whose logits are cut at every 16 of D products of which none is larger than their sum of
    absolute values.  In one term all elements move by 2^-8 |ref|, between half a step and a whole
    one: those in the upper half of a power of two leave the bound."""
    V, D = 5003, 2048
    gen = torch.Generator().manual_seed(C)
    x = (torch.randn(C, D, generator=gen) * 0.02).bfloat16()
    w = torch.randn(V, D, generator=gen).bfloat16()
    sem_row, target = np.arange(C), (np.arange(C) * 37 + 5) % V
    x64, w64 = x.double().numpy(), w.double().numpy()
    xa, wa = np.abs(x64), np.abs(w64)
    rl, re = tail.linear_logprob_fwd(x64, w64, sem_row, target)
    g = ((1 + 2.0 ** -8) / (1 - np.exp(rl))).astype(np.float32)
    row_ptr, row_sem = _csr(sem_row, C)
    dx, dw = linear_logprob_bwd(x.cuda(), w.cuda(), _dev(row_ptr), _dev(row_sem), _dev(target.astype(np.int32)),
                                _dev(re.astype(np.float32)), _dev(g))
    rdx, rdw = tail.linear_logprob_bwd(x64, w64, sem_row, target, g)
    p = np.abs(g)[:, None] * np.exp(x64 @ w64.T - re[:, None])
    own = np.zeros((C, V))
    own[sem_row, target] = np.abs(g)
    ez = D / 16 * U * (xa @ wa.T).max(axis=1) + 8 * U + U * np.abs(re)
    off = 2.0 ** -17 * (p + own) + ez[:, None] * p + 8 * U * (p + own)
    half = lambda ref: np.exp2(np.floor(np.log2(np.maximum(np.abs(ref), 1e-30))) - 8)
    at = target.tolist()
    for got, ref, bound in ((dx, rdx, off @ wa + (V / 16 + 40) * U * ((p + own) @ wa)),
                            (dw[at], rdw[at], (off.T @ xa + (C / 16 + 40) * U * ((p + own).T @ xa))[at])):
        assert np.all(np.abs(got.double().cpu().numpy() - ref) <= half(ref) + bound)
        one = np.abs(np.float64(2.0 ** -8) * ref)           # what one term would move every element by
        assert np.mean(one > half(ref) + bound) > 0.25


@pytest.mark.parametrize("C,V,D,piece", [(65_676, 1300, 136, 512), (262_129, 515, 72, 0), (262_129, 520, 64, 256)])
def test_rows_of_whole_forests(C, V, D, piece):
    """Row counts of this framework's forests, in one piece and in several, against fp64 on the GPU.
    The forward in relative L2 as above; gradients by two roundings to bf16 (dz and the result,
    2^-8 each)."""
    gen = torch.Generator(device="cuda").manual_seed(C + D)
    x = torch.randn((C, D), generator=gen, device="cuda").to(torch.bfloat16)
    w = (torch.randn((V, D), generator=gen, device="cuda") * 2 / D ** 0.5).to(torch.bfloat16)
    S = 2 * C
    sem_row = (torch.rand(S, generator=gen, device="cuda").pow(1.5) * C).long().clamp(max=C - 1)
    target = torch.randint(-1, V, (S,), generator=gen, device="cuda").to(torch.int32)
    ptr = torch.zeros(C + 1, dtype=torch.int32, device="cuda")
    ptr[1:] = torch.cumsum(torch.bincount(sem_row, minlength=C), 0)
    sem = torch.argsort(sem_row, stable=True).to(torch.int32)
    g = torch.randn(S, generator=gen, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    logp, lse = linear_logprob_fwd(x, w, ptr, sem, target, error=err)
    dx, dw = linear_logprob_bwd(x, w, ptr, sem, target, lse, g, piece=piece, error=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    z = x.double() @ w.double().t()
    re = torch.logsumexp(z, 1)
    keep, y = target >= 0, target.long().clamp(min=0)
    rl = torch.where(keep, z[sem_row, y] - re[sem_row], torch.zeros_like(re[sem_row]))
    gk = torch.where(keep, g, torch.zeros_like(g)).double()
    G = torch.zeros(C, dtype=torch.float64, device="cuda").index_add_(0, sem_row, gk)
    zmax = float(z.abs().max())
    dz = torch.exp(z - re[:, None]).mul_(-G[:, None])
    del z
    dz.index_put_((sem_row, y), gk, accumulate=True)
    u = 2.0 ** -24
    e = (0.05 * D / 16 + (D / 16) ** 0.5) * u * zmax + 8 * u
    own = ((D / 64) ** 0.5 + 8) * u * zmax
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())
    assert rel(lse, re) <= e / float(re.square().mean().sqrt()) + 2 * u
    assert rel(logp, rl) <= (e + own) / float(rl.square().mean().sqrt()) + 2 * u
    assert rel(dx, dz @ w.double()) <= 2 * 2.0 ** -8
    assert rel(dw, dz.t() @ x.double()) <= 2 * 2.0 ** -8
