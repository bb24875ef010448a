"""The operators around a recurrent layer of a rollout-tree model, as cases that can be timed and
compared.

scan: a gated linear recurrence per channel over the rows of a forest, from each row's own
predecessor on its trajectory, and its gradients.  block_norm: the norm after a block with its
gate, the residual's scaled addition and the norm before the next block in one pass, and their
gradients.  linear: a matrix product with bias, activation and residual in its epilogue, and its
gradients.  With ``own`` false the same results come from elementary torch operations in fp32
(fp64 for long sums)."""
import math
import random

import torch

own = False

CHUNK = 64                # the chunk length that this repository's plans are made with


def listed():
    """65,536-row microbatches, 2,048 channels, 16 heads of 128 and chunks of 64 are this
    repository's own; the rest are generic."""
    return [
        # decoding: 48 sequences take one step each from their states
        {"name": "scan-step", "op": "scan_fwd", "trees": 48, "segments": 48, "rows": 48, "dim": 2048, "dtype": "fp32",
         "form": "mix", "state": True},
        # a microbatch of rollout trees at its row capacity
        {"name": "scan-forest", "op": "scan_fwd", "trees": 32, "segments": 361, "rows": 65_536, "dim": 2048,
         "dtype": "bf16", "form": "add", "state": False},
        # one long trajectory: nothing but the scan's own length to work on at a time
        {"name": "scan-long", "op": "scan_fwd", "trees": 1, "segments": 1, "rows": 131_071, "dim": 1024, "dtype": "bf16",
         "form": "mix", "state": True},
        # the gradient of that microbatch
        {"name": "scan-grad-forest", "op": "scan_bwd", "trees": 32, "segments": 361, "rows": 65_536, "dim": 2048,
         "dtype": "bf16", "form": "add", "state": False},
        # the norms around a block of one sampled token: latency
        {"name": "block-norm-token", "op": "norm_fwd", "rows": 1, "dim": 2048, "dtype": "bf16", "post": True, "gate": "none",
         "residual": True, "pre": True},
        # a microbatch: norm, gate and addition after a block, norm before the next
        {"name": "block-norm-microbatch", "op": "norm_fwd", "rows": 65_536, "dim": 2048, "dtype": "bf16", "post": True,
         "gate": "silu", "residual": True, "pre": True},
        # the gated norm of every head's output behind a recurrence or an attention: short rows
        {"name": "head-norm-gate", "op": "norm_fwd", "rows": 65_535 * 16, "dim": 128, "dtype": "bf16", "post": True,
         "gate": "sigmoid", "residual": False, "pre": False},
        # the gradient of the microbatch
        {"name": "block-norm-grad-microbatch", "op": "norm_bwd", "rows": 65_536, "dim": 2048, "dtype": "bf16", "post": True,
         "gate": "silu", "residual": True, "pre": True},
        # one sampled token through a projection: reading the weight is all
        {"name": "linear-token", "op": "linear_fwd", "rows": 1, "in": 2048, "out": 8192, "act": "silu", "bias": True,
         "residual": False, "keep": False},
        # a few short branches, odd widths, back into the residual stream
        {"name": "linear-branches", "op": "linear_fwd", "rows": 777, "in": 2760, "out": 1032, "act": "none", "bias": True,
         "residual": True, "keep": False},
        # a microbatch into a wide layer, what the activation is taken of kept for the gradient
        {"name": "linear-microbatch", "op": "linear_fwd", "rows": 16_384, "in": 2048, "out": 8192, "act": "gelu",
         "bias": True, "residual": False, "keep": True},
        # the gradient of that
        {"name": "linear-grad-microbatch", "op": "linear_bwd", "rows": 16_384, "in": 2048, "out": 8192, "act": "gelu",
         "bias": True},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["scan_fwd", "scan_bwd", "norm_fwd", "norm_bwd", "linear_fwd", "linear_bwd"])
    if op in ("scan_fwd", "scan_bwd"):
        while True:
            rows, dim = _log(rng, 1, 131_071), 8 * _log(rng, 8, 512)
            dtype = rng.choice(["bf16", "bf16", "fp32"])
            if rows * dim * (2 if dtype == "fp32" else 1) <= 65_536 * 2048:
                break
        trees = min(rows, _log(rng, 1, 48))
        return {"op": op, "trees": trees, "segments": min(rows, trees * _log(rng, 1, 16)), "rows": rows, "dim": dim,
                "dtype": dtype, "form": rng.choice(["add", "mix"]), "state": rng.random() < 0.5}
    if op in ("norm_fwd", "norm_bwd"):
        while True:
            rows, dim = _log(rng, 1, 65_535 * 16), _log(rng, 64, 8191)
            if rng.random() < 0.7:
                dim = 8 * (dim // 8 | 1)
            dtype = rng.choice(["bf16", "bf16", "fp32"])
            if rows * dim * (2 if dtype == "fp32" else 1) <= 65_536 * 2048:
                break
        post, pre = rng.choice([(True, True), (True, True), (True, False), (False, True)])
        return {"op": op, "rows": rows, "dim": dim, "dtype": dtype, "post": post, "pre": pre,
                "gate": rng.choice(["none", "linear", "silu", "sigmoid"]), "residual": pre or rng.random() < 0.5}
    while True:
        c = {"op": op, "rows": _log(rng, 1, 16_384), "in": 8 * _log(rng, 16, 1024), "out": 8 * _log(rng, 16, 1024),
             "act": rng.choice(["none", "silu", "gelu"]), "bias": rng.random() < 0.7}
        if c["rows"] * c["in"] * c["out"] <= 16_384 * 2048 * 8192:
            break
    if op == "linear_fwd":
        c["residual"] = rng.random() < 0.5
        c["keep"] = rng.random() < 0.5
    return c


# ---- inputs ---------------------------------------------------------------------------------

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 1_000_003 + 29)


def _forest(case):
    """Parents and lengths of a forest's segments: a long shared prompt per tree, then branches
    that mostly go on from the newest one."""
    r = random.Random(case["rows"] * 7919 + case["segments"])
    T, n, rows = case["trees"], case["segments"], case["rows"]
    parent, newest, tree = [], list(range(T)), list(range(T))
    for i in range(n):
        if i < T:
            parent.append(-1)
            continue
        t = r.randrange(T)
        members = [j for j in range(i) if tree[j] == t]
        p = newest[t] if r.random() < 0.5 else r.choice(members)
        parent.append(p)
        tree.append(t)
        newest[t] = i
    weight = [math.exp(3 * r.random()) * (6 if p < 0 else 1) for p in parent]
    spare, total = rows - n, sum(weight)
    length = [1 + int(spare * w / total) for w in weight]
    length[0] += rows - sum(length)
    return parent, length


def _layout(parent, length):
    """Compact row of each segment's first token, as the minimum-call plan with chunks of 64 lays
    rows out: by round, then by first segment, each sequence going on into the child that needs
    most rounds itself (the lowest of several)."""
    n = len(parent)
    start, kids = [0] * n, [[] for _ in range(n)]
    for v in range(n):
        if parent[v] >= 0:
            start[v] = start[parent[v]] + length[parent[v]]
            kids[parent[v]].append(v)
    pre, into, goes_on = [1] * n, [1] * n, [-1] * n
    anchor = lambda p: p // CHUNK * CHUNK
    for v in reversed(range(n)):
        if kids[v]:
            best = max(kids[v], key=lambda c: (pre[c], -c))
            rest = max([pre[c] for c in kids[v] if c != best], default=0)
            goes_on[v], into[v] = best, max(into[best], 1 + rest)
            pre[v] = pre[best] if anchor(start[v]) == anchor(start[v] + length[v]) else into[v]
    first, when = list(range(n)), [(1, 0)] * n          # first segment of the sequence; its round and anchor
    for v in range(n):
        for c in kids[v]:
            if c == goes_on[v]:
                first[c] = first[v]
            else:
                at, (rnd, a) = anchor(start[v] + length[v]), when[first[v]]
                when[c] = (rnd, a) if at == a else (rnd + 1, at)
    offset, row, sequences = [0] * n, 0, []
    for f in sorted((v for v in range(n) if first[v] == v), key=lambda v: (when[v][0], v)):
        v = f
        while v >= 0:
            offset[v], last = row, v
            row += length[v]
            v = goes_on[v]
        sequences.append(last)
    return offset, sequences


def _rows_before(parent, length, offset):
    """For each compact row the one before it on its trajectory; -1 - r at the start of root r.
    And the number of positions before it."""
    before = torch.arange(sum(length)) - 1
    depth = torch.empty(sum(length), dtype=torch.long)
    start, root = [0] * len(parent), 0
    for v, p in enumerate(parent):
        if p < 0:
            before[offset[v]] = -1 - root
            root += 1
        else:
            before[offset[v]] = offset[p] + length[p] - 1
            start[v] = start[p] + length[p]
        depth[offset[v]:offset[v] + length[v]] = start[v] + torch.arange(length[v])
    return before.cuda(), depth.cuda()


def _scan_inputs(case, seed):
    """Log-decays as a gate gives them: channels forget within one to a thousand rows; one row in
    fifty starts afresh."""
    C, D, dt = case["rows"], case["dim"], _DT[case["dtype"]]
    parent, length = _forest(case)
    offset, sequences = _layout(parent, length)
    before, depth = _rows_before(parent, length, offset)
    g = _gen(seed)
    slow = torch.exp(-7 * torch.rand(D, generator=g, device="cuda"))
    gate = torch.rand((C, D), generator=g, device="cuda").add_(0.5).mul_(slow).neg_()
    gate[torch.rand(C, generator=g, device="cuda") < 0.02] = -30.0
    x = torch.randn((C, D), generator=g, device="cuda").to(dt)
    last = torch.tensor([offset[v] + length[v] - 1 for v in sequences], device="cuda")
    s = {"x": x, "g": gate.to(dt), "form": case["form"], "before": before, "depth": depth, "last": last, "h0": None,
         "state": case["state"], "trees": case["trees"], "steps": int(depth.max()).bit_length(),
         "parent": parent, "length": length}
    if case["state"]:
        s["h0"] = torch.randn((case["trees"], D), generator=g, device="cuda")
    return s, g


def _act(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z / math.sqrt(2.0)))
    if act == "sigmoid":
        return torch.sigmoid(z)
    return z


def _slope(z, act):
    if act == "silu":
        q = torch.sigmoid(z)
        return q * (1 + z * (1 - q))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z / math.sqrt(2.0))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "sigmoid":
        q = torch.sigmoid(z)
        return q * (1 - q)
    return torch.ones_like(z)


def prepare(case, seed):
    op = case["op"]
    if op in ("scan_fwd", "scan_bwd"):
        s, g = _scan_inputs(case, seed)
        C, D = s["x"].shape
        if op == "scan_bwd":
            s["h"] = _scan_plain(s, *_decay(s)).to(s["x"].dtype)        # the forward pass ran before
            s["dh"] = torch.randn((C, D), generator=g, device="cuda").to(s["x"].dtype)
            if s["state"]:
                s["dfinal"] = torch.randn((len(s["last"]), D), generator=g, device="cuda")
        if own:
            from prefix_shared_chunkwise_gb300.api import Plan
            s["plan"] = Plan(s["parent"], s["length"], CHUNK).upload()
        return {"op": op, **s}
    if op in ("norm_fwd", "norm_bwd"):
        C, D, dt = case["rows"], case["dim"], _DT[case["dtype"]]
        g = _gen(seed)
        rand = lambda scale: (scale * torch.randn((C, D), generator=g, device="cuda")).to(dt)
        weight = lambda: 1 + 0.2 * torch.randn(D, generator=g, device="cuda")
        s = {"op": op, "y": rand(2.0), "w_post": weight() if case["post"] else None, "w_pre": weight() if case["pre"] else None,
             "gate": rand(1.0) if case["gate"] != "none" else None, "act": case["gate"], "scale": 0.4, "eps": 1e-6,
             "res": rand(3.0) if case["residual"] else None}
        if op == "norm_bwd":                                            # the forward pass ran before
            s["h"], _, s["r_post"], s["r_pre"] = _norm_plain(s)
            s["dn"] = rand(1.0) if case["pre"] else None
            s["dh"] = rand(1.0) if case["residual"] or not case["pre"] else None
        return s
    C, K, N = case["rows"], case["in"], case["out"]
    g = _gen(seed)
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda")
    s = {"op": op, "x": rand(C, K).bfloat16(), "w": (rand(N, K) / K ** 0.5).bfloat16(), "act": case["act"],
         "b": 0.1 * rand(N) if case["bias"] else None}
    if op == "linear_fwd":
        s["res"] = rand(C, N).bfloat16() if case["residual"] else None
        s["keep"] = case["keep"]
    else:
        s["dy"] = rand(C, N).bfloat16()
        z = s["x"].float() @ s["w"].float().t()
        s["z"] = None if case["act"] == "none" else (z if s["b"] is None else z + s["b"]).bfloat16()
    return s


# ---- one pass -------------------------------------------------------------------------------

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from prefix_shared_chunkwise_gb300 import api
    op = s["op"]
    if op == "scan_fwd":
        final = None
        if s["state"]:
            final = torch.empty((len(s["last"]), s["x"].shape[1]), device="cuda")
        h = api.scan_fwd(s["plan"], s["x"], s["g"], form=s["form"], h0=s["h0"], final_state=final)
        return {"h": h, "final": final}
    if op == "scan_bwd":
        dh0 = torch.empty_like(s["h0"]) if s["state"] else None
        dx, dg = api.scan_bwd(s["plan"], s["x"], s["g"], s["h"], s["dh"], form=s["form"], h0=s["h0"],
                              d_final=s.get("dfinal"), dh0=dh0)
        return {"dx": dx, "dg": dg, "dh0": dh0}
    if op == "norm_fwd":
        h, n, r_post, r_pre = api.block_norm_fwd(s["y"], post_weight=s["w_post"], gate=s["gate"], gate_act=s["act"],
                                                 scale=s["scale"], residual=s["res"], pre_weight=s["w_pre"], eps=s["eps"])
        return {"h": h, "n": n, "r_post": r_post, "r_pre": r_pre}
    if op == "norm_bwd":
        d = api.block_norm_bwd(s["y"], s["h"], s["dn"], s["dh"], post_weight=s["w_post"], gate=s["gate"], gate_act=s["act"],
                               scale=s["scale"], pre_weight=s["w_pre"], rstd_post=s["r_post"], rstd_pre=s["r_pre"])
        return {k: d[k] for k in ("dy", "dresidual", "dgate", "dpost_weight", "dpre_weight")}
    if op == "linear_fwd":
        y, z = api.linear_fwd(s["x"], s["w"], s["b"], s["res"], activation=s["act"], keep_z=s["keep"])
        return {"y": y, "z": z}
    dx, dw, db = api.linear_bwd(s["x"], s["w"], s["dy"], s["z"], activation=s["act"], with_bias=s["b"] is not None)
    return {"dx": dx, "dw": dw, "db": db}


def _decay(s):
    """The decay and the term that is added, per row and channel."""
    g, x = s["g"].float(), s["x"].float()
    return torch.exp(g), (x if s["form"] == "add" else -torch.expm1(g) * x)


def _start(s):
    return s["h0"] if s["h0"] is not None else torch.zeros((s["trees"], s["x"].shape[1]), device="cuda")


def _scan_plain(s, a, b):
    """Pointer doubling: after k steps (a, b) spans the 2^k rows up to a row."""
    p = s["before"]
    for _ in range(s["steps"]):
        on, q = p >= 0, p.clamp(min=0)
        b = torch.where(on[:, None], b + a * b[q], b)
        a = torch.where(on[:, None], a * a[q], a)
        p = torch.where(on, p[q], p)
    return b + a * _start(s)[-1 - p]


def _scan_back_plain(s, a, u):
    """The sums over what follows a row, u the gradients that arrive at it from outside: after k
    steps u spans the rows up to 2^k positions behind it and c the decays of a row and those
    before it back to p."""
    p, c = s["before"], a
    for _ in range(s["steps"]):
        on, q = p >= 0, p.clamp(min=0)
        u = u.index_add(0, q, torch.where(on[:, None], c * u, torch.zeros_like(u)))
        c = torch.where(on[:, None], c * c[q], c)
        p = torch.where(on, p[q], p)
    return u


def _norm_plain(s):
    v, dt, r_post, r_pre, n = s["y"].float(), s["y"].dtype, None, None, None
    if s["w_post"] is not None:
        r_post = torch.rsqrt(v.square().mean(1) + s["eps"])
        v = v * r_post[:, None] * s["w_post"]
    if s["gate"] is not None:
        v = v * _act(s["gate"].float(), s["act"])
    h = s["scale"] * v
    if s["res"] is not None:
        h = h + s["res"].float()
    if s["w_pre"] is not None:
        r_pre = torch.rsqrt(h.square().mean(1) + s["eps"])
        n = (h * r_pre[:, None] * s["w_pre"]).to(dt)
    return h.to(dt), n, r_post, r_pre


def _run_plain(s):
    op = s["op"]
    if op == "scan_fwd":
        h = _scan_plain(s, *_decay(s))
        return {"h": h.to(s["x"].dtype), "final": h[s["last"]] if s["state"] else None}
    if op == "scan_bwd":
        a, _ = _decay(s)
        u = s["dh"].float()
        if s["state"]:
            u = u.index_add(0, s["last"], s["dfinal"])
        lam = _scan_back_plain(s, a, u)
        p = s["before"]
        prev = torch.where((p >= 0)[:, None], s["h"].float()[p.clamp(min=0)], _start(s)[(-1 - p).clamp(min=0)])
        if s["form"] == "add":
            dx, dg = lam, lam * a * prev
        else:
            dx, dg = lam * -torch.expm1(s["g"].float()), lam * a * (prev - s["x"].float())
        dh0 = None
        if s["state"]:
            first = (p < 0).nonzero()[:, 0]
            dh0 = torch.zeros_like(s["h0"]).index_add(0, -1 - p[first], a[first] * lam[first])
        return {"dx": dx.to(s["x"].dtype), "dg": dg.to(s["x"].dtype), "dh0": dh0}
    if op == "norm_fwd":
        h, n, r_post, r_pre = _norm_plain(s)
        return {"h": h, "n": n, "r_post": r_post, "r_pre": r_pre}
    if op == "norm_bwd":
        dt, out = s["y"].dtype, dict.fromkeys(("dy", "dresidual", "dgate", "dpost_weight", "dpre_weight"))
        d = s["dh"].float() if s["dh"] is not None else 0.0
        if s["w_pre"] is not None:
            dn, r = s["dn"].float(), s["r_pre"][:, None]
            n = s["h"].float() * r
            t = dn * s["w_pre"]
            d = r * (t - n * (t * n).mean(1, keepdim=True)) + d
            out["dpre_weight"] = (dn * n).sum(0, dtype=torch.float64).float()
            out["dresidual"] = d.to(dt)
        y = s["y"].float()
        u = y if s["w_post"] is None else y * s["r_post"][:, None] * s["w_post"]
        du = s["scale"] * d
        if s["gate"] is not None:
            z = s["gate"].float()
            out["dgate"] = (du * u * _slope(z, s["act"])).to(dt)
            du = du * _act(z, s["act"])
        if s["w_post"] is not None:
            r = s["r_post"][:, None]
            n, t = y * r, du * s["w_post"]
            out["dpost_weight"] = (du * n).sum(0, dtype=torch.float64).float()
            du = r * (t - n * (t * n).mean(1, keepdim=True))
        out["dy"] = du.to(dt)
        return out
    if op == "linear_fwd":
        z = s["x"].float() @ s["w"].float().t()
        if s["b"] is not None:
            z = z + s["b"]
        y = _act(z, s["act"])
        if s["res"] is not None:
            y = y + s["res"].float()
        return {"y": y.bfloat16(), "z": z.bfloat16() if s["keep"] else None}
    dz = s["dy"].float()
    if s["z"] is not None:
        dz = dz * _slope(s["z"].float(), s["act"])
    return {"dx": (dz @ s["w"].float()).bfloat16(), "dw": (dz.t() @ s["x"].float()).bfloat16(),
            "db": dz.sum(0, dtype=torch.float64).float() if s["b"] is not None else None}


# ---- what a pass cannot do without ----------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("scan_fwd", "scan_bwd"):
        n, size = case["rows"] * case["dim"], 2 if case["dtype"] == "bf16" else 4
        states = 0
        if case["state"]:
            parent, length = _forest(case)
            inner = {p for p in parent if p >= 0}
            states = 4 * case["dim"] * (case["trees"] + len(parent) - len(inner))
            if op == "scan_bwd":
                states += 4 * case["dim"] * case["trees"]               # both h0 and its gradient
        if op == "scan_fwd":
            return {"bytes": 3 * size * n + states, "flops": 3 * n}
        # with the addition x itself has no part in the gradients
        return {"bytes": size * n * (5 if case["form"] == "add" else 6) + states, "flops": 8 * n}
    if op in ("norm_fwd", "norm_bwd"):
        n, size = case["rows"] * case["dim"], 2 if case["dtype"] == "bf16" else 4
        gate, res, norms = case["gate"] != "none", case["residual"], case["post"] + case["pre"]
        if op == "norm_fwd":
            streams = 2 + gate + res + case["pre"]
            return {"bytes": n * size * streams + norms * (4 * case["dim"] + 4 * case["rows"]), "flops": 12 * n}
        streams = 2 + 2 * gate                                          # y, its gradient; the gate and its
        streams += 3 * case["pre"]                                      # h, dn and the residual's gradient
        streams += 1 if res or not case["pre"] else 0                   # dh
        return {"bytes": n * size * streams + norms * (8 * case["dim"] + 4 * case["rows"]), "flops": 24 * n}
    C, K, N = case["rows"], case["in"], case["out"]
    if op == "linear_fwd":
        out = 2 * C * N * (1 + case["residual"] + case["keep"]) + 4 * N * case["bias"]
        return {"bytes": 2 * K * (C + N) + out, "flops": 2 * C * K * N}
    return {"bytes": 4 * K * (C + N) + 2 * C * N * (2 if case["act"] != "none" else 1) + 4 * N * case["bias"],
            "flops": 4 * C * K * N}


# ---- the definitions in 64 bits -------------------------------------------------------------

def _by_depth(depth):
    order = torch.argsort(depth, stable=True)
    return order, torch.bincount(depth).tolist()


def _gate64(z, kind):
    """A gate's or an activation's value and derivative."""
    z = z.double()
    if kind in ("silu", "sigmoid"):
        q = 1 / (1 + torch.exp(-z))
        dq = q * torch.exp(-z) / (1 + torch.exp(-z))
        dq = torch.where(z < -700, torch.zeros_like(z), dq)
        return (q, dq) if kind == "sigmoid" else (z * q, q + z * dq)
    if kind == "gelu":
        cdf = 0.5 * torch.erfc(-z * 0.7071067811865476)
        return z * cdf, cdf + z * torch.exp(-z * z / 2) * 0.3989422804014327
    return z, torch.ones_like(z)


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op in ("scan_fwd", "scan_bwd"):
        # one position of every trajectory after another
        g, p = s["g"].double(), s["before"]
        order, counts = _by_depth(s["depth"])
        D, trees = g.shape[1], case["trees"]
        start = s["h0"].double() if s["state"] else torch.zeros((trees, D), dtype=torch.float64, device="cuda")
        a = torch.exp(g)
        keep = 1 - a if s["form"] == "mix" else torch.ones_like(a)
        small = g.abs() < 1e-5
        if s["form"] == "mix":
            keep = torch.where(small, -g - g * g / 2, keep)
        spans, at = [], 0
        for n in counts:
            spans.append(order[at:at + n])
            at += n
        if op == "scan_fwd":
            h = keep * s["x"].double()
            rows = spans[0]
            h[rows] += a[rows] * start[-1 - p[rows]]
            if max(counts) == 1 and bool((order[1:] == order[:-1] + 1).all()):
                for t in range(1, len(h)):
                    h[t].addcmul_(a[t], h[t - 1])
            else:
                for rows in spans[1:]:
                    h[rows] += a[rows] * h[p[rows]]
            return {"h": h, "final": h[s["last"]] if s["state"] else None}
        lam = s["dh"].double()
        if s["state"]:
            lam[s["last"]] += s["dfinal"].double()
        for rows in reversed(spans[1:]):
            lam.index_put_((p[rows],), a[rows] * lam[rows], accumulate=True)
        prev = torch.empty_like(lam)
        inner = p >= 0
        prev[inner] = s["h"].double()[p[inner]]
        prev[~inner] = start[-1 - p[~inner]]
        dg = lam * a * (prev - s["x"].double() if s["form"] == "mix" else prev)
        dh0 = None
        if s["state"]:
            dh0 = torch.empty_like(start)
            dh0[-1 - p[spans[0]]] = a[spans[0]] * lam[spans[0]]
        return {"dx": keep * lam, "dg": dg, "dh0": dh0}
    if op == "norm_fwd":
        y = s["y"].double()
        r_post = r_pre = n = None
        if s["w_post"] is not None:
            r_post = ((y * y).sum(1) / y.shape[1] + s["eps"]).pow(-0.5)
            y = y * r_post.unsqueeze(1) * s["w_post"].double()
        h = s["scale"] * y * (_gate64(s["gate"], s["act"])[0] if s["gate"] is not None else 1.0)
        if s["res"] is not None:
            h = h + s["res"].double()
        if s["w_pre"] is not None:
            r_pre = ((h * h).sum(1) / h.shape[1] + s["eps"]).pow(-0.5)
            n = h * r_pre.unsqueeze(1) * s["w_pre"].double()
        return {"h": h, "n": n, "r_post": r_post, "r_pre": r_pre}
    if op == "norm_bwd":
        # h and the two reciprocal roots are inputs here, as the forward pass left them
        D = s["y"].shape[1]
        out = dict.fromkeys(("dy", "dresidual", "dgate", "dpost_weight", "dpre_weight"))
        into = s["dh"].double() if s["dh"] is not None else torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
        if s["w_pre"] is not None:
            h, dn, r = s["h"].double(), s["dn"].double(), s["r_pre"].double().unsqueeze(1)
            w = s["w_pre"].double()
            into = into + dn * w * r - h * r.pow(3) * ((dn * w * h).sum(1, keepdim=True) / D)
            out["dpre_weight"] = (dn * h * r).sum(0)
            out["dresidual"] = into
        y, value, slope = s["y"].double(), 1.0, None
        if s["gate"] is not None:
            value, slope = _gate64(s["gate"], s["act"])
        if s["w_post"] is None:
            normed, out["dy"] = y, s["scale"] * into * value
        else:
            w, r = s["w_post"].double(), s["r_post"].double().unsqueeze(1)
            normed, t = y * r * w, s["scale"] * into * value
            out["dpost_weight"] = (t * y * r).sum(0)
            out["dy"] = t * w * r - y * r.pow(3) * ((t * w * y).sum(1, keepdim=True) / D)
        if slope is not None:
            out["dgate"] = s["scale"] * into * normed * slope
        return out
    x, w = s["x"].double(), s["w"].double()
    if op == "linear_fwd":
        z = torch.matmul(x, w.T)
        if s["b"] is not None:
            z += s["b"].double()
        y = _gate64(z, s["act"])[0]
        if s["res"] is not None:
            y = y + s["res"].double()
        return {"y": y, "z": z if s["keep"] else None}
    dz = s["dy"].double()
    if s["z"] is not None:
        dz = dz * _gate64(s["z"], s["act"])[1]
    return {"dx": torch.matmul(dz, w), "dw": torch.matmul(dz.T, x), "db": dz.sum(0) if s["b"] is not None else None}
