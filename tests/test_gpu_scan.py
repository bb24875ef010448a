"""GPU parity of harts_scan_fwd / _bwd against the fp64 oracle (oracle/scan.py) on the same (cast)
inputs, element by element.

Bounds.  u = 2^-24 (fp32 half step), r half a step of the output type relative to the value.  A
decay is within 4 u of e^g (series, its rounding, 1 - a and back); a row adds one fused
product and sum, one product of decays, and its share of the joins (one in 16 rows, one in 128):
at most 12 u of a S + |b| in all, S the same recurrence over absolute values, and what a row is off
by is carried on like the state: E = a E_before + 12 u (a S_before + |b|).  bf16 results of the add
form take the hardware's exponential, 2^-22 or 4 u, of a product that is off by |g| u: 16 u more, and
a |g| <= 1/e of them.  The mix form's forward takes a from 1 - a, which leaves it off by 2^-25 however
small it is: u S_before more.  The backward's lam goes the same way from the leaves, and dx, dg are products
of it with up to four roundings more."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle.scan import scan_forest, scan_forest_bwd
from prefix_shared_chunkwise_gb300.api import Plan, scan_bwd, scan_fwd

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": (torch.bfloat16, 2.0 ** -8), "fp32": (torch.float32, U)}
K = {"bf16": 28, "fp32": 12}

# one row, a chain, forks inside and at the end of a tile, fans, deep chains of short segments
FORESTS = {
    "one-row": ([-1], [1]),
    "one-tile": ([-1], [128]),
    "just-over": ([-1, 0], [129, 1]),
    "chain": ([-1], [700]),
    "groups": ([-1], [2 * 4096 + 77]),                                  # three groups of tiles
    "group-ends": ([-1, 0, 0, 2], [4096, 4096, 4097, 3]),
    "fork": ([-1, 0, 0, 1, 1, 2], [100, 50, 70, 90, 40, 1]),
    "fan": ([-1] + [0] * 40, [37] + [1 + 5 * i for i in range(40)]),
    "deep": ([-1] + list(range(60)), [1 + (7 * i) % 23 for i in range(61)]),
    "trees": ([-1, -1, -1, 0, 1, 1, 5, 3, 3], [1, 200, 16, 129, 15, 257, 64, 2, 300]),
    "roots": ([-1] * 9, [1, 128, 17, 5, 64, 100, 3, 2, 99]),            # no tile follows another
    "steps": ([-1] * 13, [1] * 13),                                     # a decoding step
}


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from prefix_shared_chunkwise_gb300 import build
    build.build()


def _np(t):
    return t.double().cpu().numpy()


def plan_bytes(plan, D):
    from prefix_shared_chunkwise_gb300 import _lib as L
    return L.lib().harts_scan_workspace_bytes(plan.handle, D, L.HARTS_BF16)


class Case:
    def __init__(self, forest, D, dtype, form, state, seed=0, **plan):
        self.parent, self.len = forest
        self.plan = Plan(self.parent, self.len, 64, **plan).upload()
        self.arr = self.plan.arrays()
        self.off = [int(o) for o in self.arr["seg_offset"]]
        self.form, self.dtype = form, dtype
        td, self.r = DT[dtype]
        C = self.plan.info["C"]
        g = torch.Generator().manual_seed(seed + C)
        slow = torch.exp(-7 * torch.rand(D, generator=g))
        self.x = torch.randn((C, D), generator=g).to(td).cuda()
        gate = -(torch.rand((C, D), generator=g) + 0.5) * slow
        gate[torch.rand(C, generator=g) < 0.02] = -30.0
        gate[torch.rand((C, D), generator=g) < 0.01] = 0.0
        gate[torch.rand((C, D), generator=g) < 0.005] = -torch.inf
        self.g = gate.to(td).cuda()
        self.dh = torch.randn((C, D), generator=g).to(td).cuda()
        info = self.plan.info
        self.h0 = torch.randn((info["n_roots"], D), generator=g).cuda() if state else None
        self.dfinal = torch.randn((info["n_seq"], D), generator=g).cuda() if state else None
        self.last = [int(e) - 1 for e in self.arr["cu_seqlens"][1:]]
        self.state = state

    def forward(self, **kw):
        final = torch.full_like(self.dfinal, 7.0) if self.state else None
        return scan_fwd(self.plan, self.x, self.g, form=self.form, h0=self.h0, final_state=final, **kw), final

    def backward(self, h, **kw):
        dh0 = torch.full_like(self.h0, 7.0) if self.state else None
        return (*scan_bwd(self.plan, self.x, self.g, h, self.dh, form=self.form, h0=self.h0, d_final=self.dfinal, dh0=dh0,
                          **kw), dh0)

    def check_forward(self):
        h, final = self.forward()
        torch.cuda.synchronize()
        assert self.plan.device_error() == 0
        x, g, mix = _np(self.x), _np(self.g), self.form == "mix"
        h0 = None if self.h0 is None else _np(self.h0)
        ref, prev = scan_forest(self.parent, self.len, self.off, x, g, mix, h0)
        b = np.abs(-np.expm1(g) * x if mix else x)
        size, before = scan_forest(self.parent, self.len, self.off, b, g, False, None if h0 is None else np.abs(h0))
        step = K[self.dtype] * U
        own = U * before if mix else 0.0
        err, _ = scan_forest(self.parent, self.len, self.off, step * (np.exp(g) * before + b) + own, g, False)
        assert np.all(np.abs(_np(h) - ref) <= self.r * np.abs(ref) + err + 1e-37)
        if self.state:
            err, _ = scan_forest(self.parent, self.len, self.off, 12 * U * (np.exp(g) * before + b) + own, g, False)
            assert np.all(np.abs(_np(final) - ref[self.last]) <= err[self.last] + 1e-37)
        return h

    def check_backward(self, h):
        dx, dg, dh0 = self.backward(h)
        torch.cuda.synchronize()
        assert self.plan.device_error() == 0
        x, g, mix, hn, d = _np(self.x), _np(self.g), self.form == "mix", _np(h), _np(self.dh)
        h0 = None if self.h0 is None else _np(self.h0)
        prev = np.empty_like(hn)
        root = 0
        for v, p in enumerate(self.parent):
            o = self.off[v]
            if p >= 0:
                prev[o] = hn[self.off[p] + self.len[p] - 1]
            else:
                prev[o] = 0 if h0 is None else h0[root]
                root += 1
            prev[o + 1:o + self.len[v]] = hn[o:o + self.len[v] - 1]
        ends = None if self.dfinal is None else {r: _np(self.dfinal)[i] for i, r in enumerate(self.last)}
        args = (self.parent, self.len, self.off, x, g, mix, prev)
        rdx, rdg, rdh0, lam = scan_forest_bwd(*args, d, h0, ends)
        up = None if ends is None else {r: np.abs(e) for r, e in ends.items()}
        _, _, s0, size = scan_forest_bwd(self.parent, self.len, self.off, x, g, False, prev, np.abs(d), h0, up)
        k = K[self.dtype]
        _, _, e0, err = scan_forest_bwd(self.parent, self.len, self.off, x, g, False, prev, k * U * size, h0, None)
        a, om = np.exp(g), -np.expm1(g)
        assert np.all(np.abs(_np(dx) - rdx) <= self.r * np.abs(rdx) + (om if mix else 1) * (err + 4 * U * size) + 1e-37)
        q = a * np.abs(prev - x if mix else prev)
        assert np.all(np.abs(_np(dg) - rdg) <= self.r * np.abs(rdg) + q * (err + 4 * U * size)
                      + 4 * U * a * size * (np.abs(prev) + (np.abs(x) if mix else 0)) + 1e-37)
        if self.state:
            assert np.all(np.abs(_np(dh0) - rdh0) <= 12 / k * e0 + 4 * U * s0 + 1e-37)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("form,state", [("add", False), ("mix", True)])
@pytest.mark.parametrize("forest", sorted(FORESTS))
def test_forests(forest, form, state, dtype):
    c = Case(FORESTS[forest], 72, dtype, form, state)
    c.check_backward(c.check_forward())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D", [8, 24, 32, 64, 136, 264])
def test_channels(D, dtype):
    for form, state in (("add", True), ("mix", False)):
        c = Case(FORESTS["trees"], D, dtype, form, state, seed=D)
        c.check_backward(c.check_forward())


@pytest.mark.parametrize("plan", [dict(nodewise=True), dict(noreplay=True)])
def test_plan_modes(plan):
    for dtype in ("bf16", "fp32"):
        c = Case(FORESTS["trees"], 40, dtype, "mix", True, seed=5, **plan)
        c.check_backward(c.check_forward())


@pytest.mark.parametrize("name", ["fig1_fp32", "fwd16k_bf16"])
def test_rollout_forests(name):
    from prefix_shared_chunkwise_gb300.synth import make_tree
    parent, seg_len = make_tree(name)
    c = Case(([int(p) for p in parent], [int(n) for n in seg_len]), 64, "bf16", "mix", True, seed=1)
    c.check_backward(c.check_forward())


def test_same_bits_on_every_run_and_whatever_the_workspace_held():
    c = Case(FORESTS["groups"], 1000, "bf16", "add", True)
    from prefix_shared_chunkwise_gb300 import _lib
    nb = _lib.lib().harts_scan_workspace_bytes(c.plan.handle, 1000, 1)
    first = None
    for fill in (0, 0xff, 0x7f, 1):
        ws = torch.full((nb,), fill, dtype=torch.uint8, device="cuda")
        h, final = c.forward(workspace=ws)
        out = [h, final, *c.backward(h, workspace=ws)]
        first = first or out
        assert all(torch.equal(a, b) for a, b in zip(first, out))


def test_what_is_not_finite_stays_on_its_trajectories():
    forest = ([-1, 0, 0, -1, 2], [140, 150, 20, 130, 9])
    c = Case(forest, 64, "fp32", "add", False)
    c.g.clamp_(min=-0.5)
    h, _ = c.forward()
    dx, dg, _ = c.backward(h)
    row = c.off[2] + 5                                    # inside segment 2, before segment 4
    c.x[row, 3] = float("nan")
    h2, _ = c.forward()
    behind = torch.zeros(c.x.shape[0], dtype=torch.bool, device="cuda")
    behind[row:c.off[2] + 20] = True
    behind[c.off[4]:c.off[4] + 9] = True
    assert bool(h2[behind, 3].isnan().all())
    same = (h2 == h)
    same[behind, 3] = True
    assert bool(same.all())
    c.dh[row, 4] = float("inf")                           # backward: the rows before it
    dx2, dg2, _ = c.backward(h)
    before = torch.zeros_like(behind)
    before[c.off[2]:row + 1] = True
    before[c.off[0]:c.off[0] + 140] = True
    assert not bool(dx2[before, 4].isfinite().any())
    same = (dx2 == dx)
    same[before, 4] = True
    assert bool(same.all())


def test_h0_of_one_step_is_a_row_of_a_longer_scan():
    """Decoding: a scan of 20 rows, and the same rows one step at a time from the states before."""
    B, T, D = 5, 20, 48
    long = Plan([-1] * B, [T] * B, 64).upload()
    step = Plan([-1] * B, [1] * B, 64).upload()
    gen = torch.Generator().manual_seed(3)
    x, g = torch.randn(B, T, D, generator=gen).cuda(), -torch.rand(B, T, D, generator=gen).cuda()
    final = torch.empty(B, D, device="cuda")
    h = scan_fwd(long, x.view(B * T, D), g.view(B * T, D), form="mix", final_state=final).view(B, T, D)
    state = torch.zeros(B, D, device="cuda")
    for t in range(T):
        out = scan_fwd(step, x[:, t].contiguous(), g[:, t].contiguous(), form="mix", h0=state, final_state=state)
        assert torch.equal(out, state)
        # two orders of joining at most 20 rows: 12 u a row of values whose sizes add up to at most T
        assert float((out - h[:, t]).abs().max()) <= 2 * 12 * U * T * 4
    assert float((state - final).abs().max()) <= 2 * 12 * U * T * 4


def test_captured_and_on_another_stream():
    c = Case(FORESTS["trees"], 264, "bf16", "mix", True, seed=9)
    h, final = c.forward()
    want = [h, final, *c.backward(h)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    h2, f2 = c.forward(stream=s)
    got = [h2, f2, *c.backward(h2, stream=s)]
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h3, f3 = c.forward()
        out = [h3, f3, *c.backward(h3)]
    x = c.x.clone()
    for _ in range(2):
        c.x.neg_()
        graph.replay()
        c.x.copy_(x)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, out))
    assert c.plan.device_error() == 0



LONG = {
    "chain": ([-1], [9001]),
    "forks": ([-1, 0, 0, 1, 1, 4, -1, 6], [5000, 300, 2100, 2048, 4096, 129, 1, 8200]),
    "short-segments": ([-1] + list(range(89)), [1 + (37 * i) % 200 for i in range(90)]),
}


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("form,state", [("add", False), ("mix", True), ("add", True)])
@pytest.mark.parametrize("D", [40, 264])
@pytest.mark.parametrize("forest", sorted(LONG))
def test_long_trajectories(forest, D, form, state, dtype):
    c = Case(LONG[forest], D, dtype, form, state)
    assert sum(c.len) >= 8192
    h = c.check_forward()
    c.check_backward(h)
    assert torch.equal(h.view(torch.uint8), c.forward()[0].view(torch.uint8))


def test_slow_decays_over_a_long_trajectory():
    """x = 1 and a decay per channel that stays: h_t = (1 - a^(t+1)) / (1 - a).  A row adds half a u for a
    (a rounded number below 1), one for the product of decays and as much for the sum, of which 1 in 16, 1 in
    128 and 1 in 4,096 rows have more: 1.7 u in all, once for every row that a term is old."""
    T, D = 131_072, 64
    plan = Plan([-1], [T], 64).upload()
    g = -torch.exp(torch.linspace(-4, -15, D)).bfloat16()
    x = torch.ones(T, D, dtype=torch.bfloat16, device="cuda")
    h = scan_fwd(plan, x, g.cuda().expand(T, D).contiguous())
    torch.cuda.synchronize()
    assert plan.device_error() == 0
    n, lg = np.arange(1, T + 1)[:, None], _np(g)[None]
    ref = np.expm1(n * lg) / np.expm1(lg)
    a = np.exp(lg)
    age = a / -np.expm1(lg) - n * np.exp(n * lg) / -np.expm1(n * lg)        # of a term, by its share of the sum
    assert np.all(np.abs(_np(h) - ref) <= (2.0 ** -8 + 1.7 * U * (age + 1)) * ref)


def test_long_trajectories_captured_and_two_at_once():
    """Blocks of two calls wait for their own call's blocks only."""
    c = [Case(LONG["forks"], 264, "bf16", "mix", True, seed=s) for s in (1, 2)]
    plan = c[0].plan
    want = [x.forward() for x in c]
    back = [x.backward(h) for x, (h, _) in zip(c, want)]
    ws = [torch.empty(plan_bytes(plan, 264), dtype=torch.uint8, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs, got = [], []
    for x, w, st in zip(c, ws, streams):
        h, final = torch.empty_like(want[0][0]), torch.empty_like(want[0][1])
        dx, dg, dh0 = torch.empty_like(h), torch.empty_like(h), torch.empty_like(x.h0)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            scan_fwd(plan, x.x, x.g, form="mix", h0=x.h0, final_state=final, h=h, workspace=w)
            scan_bwd(plan, x.x, x.g, h, x.dh, form="mix", h0=x.h0, d_final=x.dfinal, dx=dx, dg=dg, dh0=dh0, workspace=w)
        graphs.append(graph)
        got.append((h, final, dx, dg, dh0))
    for _ in range(4):
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    assert plan.device_error() == 0
    for g, w, b in zip(got, want, back):
        for a, e in zip(g, (*w, *b)):
            assert torch.equal(a, e)
