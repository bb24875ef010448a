"""The operators of an update step's tail, as cases that can be timed and compared.

linear_logprob: log-probabilities of semantic positions from hidden rows and the vocabulary
weight, without kept logits, and their gradients.  rmsnorm: the residual's addition and the
norm before it, forward (bf16 / fp32 / 8-bit blocks) and backward.  grad_clip: the norm over
all gradients, and clipping.  With ``own`` false the same results come from elementary torch
operations in fp32 (fp64 for long sums)."""
import torch

own = False

V_FULL = 157_184          # the vocabulary of the log-probability workload
BLOCK = 32                # channels that share one scale in the 8-bit form


def listed():
    """Sizes: the vocabulary 157,184 and 65,536-row microbatches are this repository's own;
    the rest are generic."""
    return [
        # one sampled token is scored against the full vocabulary: reading the weight is all
        {"name": "head-one-token", "op": "head_fwd", "rows": 1, "vocab": V_FULL, "dim": 2048},
        # a few short branches with a small, odd vocabulary and an odd width
        {"name": "head-short-branches", "op": "head_fwd", "rows": 777, "vocab": 32_003, "dim": 1032},
        # the compact rows of one forest
        {"name": "head-forest", "op": "head_fwd", "rows": 4096, "vocab": V_FULL, "dim": 2048},
        # the gradient of one short branch
        {"name": "head-grad-branch", "op": "head_bwd", "rows": 61, "vocab": 32_003, "dim": 1032},
        # the gradient of one forest
        {"name": "head-grad-forest", "op": "head_bwd", "rows": 4096, "vocab": V_FULL, "dim": 2048},
        # the norm of one sampled token: latency
        {"name": "norm-one-token", "op": "norm_fwd", "rows": 1, "dim": 2048, "dtype": "bf16", "residual": True,
         "mx8": False},
        # a microbatch at its row capacity
        {"name": "norm-microbatch", "op": "norm_fwd", "rows": 65_536, "dim": 2048, "dtype": "bf16",
         "residual": True, "mx8": False},
        # the norm that feeds an 8-bit projection
        {"name": "norm-mx8", "op": "norm_fwd", "rows": 8191, "dim": 4096, "dtype": "bf16", "residual": True,
         "mx8": True},
        # fp32 rows of an odd width (no row is aligned)
        {"name": "norm-grad-odd-fp32", "op": "norm_bwd", "rows": 1237, "dim": 1001, "dtype": "fp32",
         "residual": False},
        # the gradient of a microbatch, with the residual stream's own gradient
        {"name": "norm-grad-microbatch", "op": "norm_bwd", "rows": 65_536, "dim": 2048, "dtype": "bf16",
         "residual": True},
        # adapters or one small layer: a few tensors of odd sizes and both types
        {"name": "clip-small", "op": "clip", "tensors": 23, "values": 1_000_003, "dtype": "mixed"},
        # a model's bf16 gradients: one large embedding, matrices and many small vectors
        {"name": "clip-model", "op": "clip", "tensors": 61, "values": 600_000_000, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["head_fwd", "head_bwd", "norm_fwd", "norm_bwd", "clip"])
    if op in ("head_fwd", "head_bwd"):
        most = 4096 * V_FULL * 2048
        while True:
            c = {"op": op, "rows": _log(rng, 1, 4096) | 1, "vocab": _log(rng, 1000, V_FULL - 2) | 1,
                 "dim": 8 * (_log(rng, 32, 500) | 1)}
            if c["rows"] * c["vocab"] * c["dim"] <= most and c["vocab"] * c["dim"] <= V_FULL * 2048:
                return c
    if op in ("norm_fwd", "norm_bwd"):
        while True:
            rows, dim = _log(rng, 1, 65_535) | 1, _log(rng, 64, 8191)
            if rows * dim <= 65_536 * 2048:
                break
        dtype, residual = rng.choice(["bf16", "bf16", "fp32"]), rng.random() < 0.7
        if rng.random() < 0.5:
            dim = 8 * (dim // 8 | 1)
        if dtype == "fp32":
            rows = (rows + 1) // 2 | 1
        c = {"op": op, "rows": rows, "dim": dim, "dtype": dtype, "residual": residual}
        if op == "norm_fwd":
            c["mx8"] = rng.random() < 0.3
            if c["mx8"]:
                c["rows"], c["dim"] = min(rows, 8191), BLOCK * (dim // BLOCK | 1)
        return c
    dtype = rng.choice(["bf16", "fp32", "mixed"])
    return {"op": "clip", "tensors": _log(rng, 1, 60), "values": _log(rng, 1000, 300_000_000) | 1, "dtype": dtype}


# ---- inputs ---------------------------------------------------------------------------------

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 1_000_003 + 17)


def _positions(rows):
    return 3 * rows if rows > 1 else 1


def _head_inputs(case, seed):
    """Hidden rows as a norm leaves them, a weight that gives logits a spread of about 2, and
    labels that the rows favour, as sampled tokens are.  Three semantic positions a row on
    average: rows near a trajectory's end have one or none, shared prefix rows many; positions
    of one row mostly share their label and differ at forks; one in a hundred has none (-1)."""
    C, V, D = case["rows"], case["vocab"], case["dim"]
    g = _gen(seed)
    w = torch.empty((V, D), dtype=torch.bfloat16, device="cuda")
    w.normal_(0.0, 2.0 / D ** 0.5, generator=g)
    main = torch.randint(0, V, (C,), generator=g, device="cuda")
    pull = torch.rand((C, 1), generator=g, device="cuda") * 4
    x = (torch.randn((C, D), generator=g, device="cuda") + pull * w[main].float()).to(torch.bfloat16)
    S = _positions(C)
    sem_row = (torch.rand(S, generator=g, device="cuda").pow(1.5) * C).long().clamp(max=C - 1)
    other = torch.randint(0, V, (S,), generator=g, device="cuda")
    u = torch.rand(S, generator=g, device="cuda")
    target = torch.where(u < 0.9, main[sem_row], other)
    target = torch.where(u > 0.99, torch.full_like(target, -1), target).to(torch.int32)
    row_ptr = torch.zeros(C + 1, dtype=torch.int32, device="cuda")
    row_ptr[1:] = torch.cumsum(torch.bincount(sem_row, minlength=C), 0)
    row_sem = torch.argsort(sem_row, stable=True).to(torch.int32)
    return {"x": x, "w": w, "sem_row": sem_row, "row_ptr": row_ptr, "row_sem": row_sem, "target": target, "g": g}


def _norm_inputs(case, seed):
    C, D, dt = case["rows"], case["dim"], _DT[case["dtype"]]
    g = _gen(seed)
    weight = 1 + 0.2 * torch.randn(D, generator=g, device="cuda")
    a = torch.randn((C, D), generator=g, device="cuda").to(dt)
    b = (3 * torch.randn((C, D), generator=g, device="cuda")).to(dt) if case["residual"] else None
    return g, weight, a, b


def _clip_sizes(case):
    """One tensor with half of the values, then matrices and vectors, odd sizes among them."""
    n, total = case["tensors"], case["values"]
    if n == 1:
        return [total]
    r = torch.Generator().manual_seed(n)
    part = torch.exp(torch.rand(n - 1, generator=r) * 6)
    part = (part / part.sum() * (total - total // 2)).long().clamp(min=1).tolist()
    return [total // 2] + [p if i % 3 == 0 else (p + 7) // 8 * 8 for i, p in enumerate(part)]


def prepare(case, seed):
    op = case["op"]
    if op in ("head_fwd", "head_bwd"):
        s = _head_inputs(case, seed)
        g = s.pop("g")
        if op == "head_bwd":
            S = s["target"].numel()
            adv = torch.randn(S, generator=g, device="cuda") / max(S, 1)
            s["dlogp"] = torch.where(torch.rand(S, generator=g, device="cuda") < 0.3, torch.zeros_like(adv), adv)
            parts = [_lse(z) for z in (s["x"][i:i + 512].float() @ s["w"].float().t()
                                       for i in range(0, case["rows"], 512))]
            s["lse"] = torch.cat(parts)             # the forward pass ran before
        return {"op": op, **s}
    if op == "norm_fwd":
        _, weight, x, res = _norm_inputs(case, seed)
        return {"op": op, "x": x, "res": res, "weight": weight, "eps": 1e-6, "mx8": case["mx8"]}
    if op == "norm_bwd":
        g, weight, dy, h = _norm_inputs(dict(case, residual=True), seed)
        rstd = torch.rsqrt(h.double().square().mean(1) + 1e-6).float()
        dh = torch.randn(h.shape, generator=g, device="cuda").to(h.dtype) if case["residual"] else None
        return {"op": op, "dy": dy, "h": h, "dh": dh, "weight": weight, "rstd": rstd}
    g = _gen(seed)
    kinds = {"bf16": [torch.bfloat16], "fp32": [torch.float32], "mixed": [torch.bfloat16, torch.float32]}[case["dtype"]]
    grads = [(torch.randn(n, generator=g, device="cuda") * 1e-3).to(kinds[i % len(kinds)])
             for i, n in enumerate(_clip_sizes(case))]
    s = {"op": op, "grads": grads, "max_norm": 0.37e-3 * case["values"] ** 0.5,
         "out": [torch.empty_like(t) for t in grads]}
    if own:                                          # a program makes the set once for its buffers
        from prefix_shared_chunkwise_gb300.api import GradSet
        s["set"] = GradSet(s["grads"], s["out"])
    return s


# ---- one pass -------------------------------------------------------------------------------

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from prefix_shared_chunkwise_gb300 import api
    op = s["op"]
    if op == "head_fwd":
        logp, lse = api.linear_logprob_fwd(s["x"], s["w"], s["row_ptr"], s["row_sem"], s["target"])
        return {"logp": logp, "lse": lse}
    if op == "head_bwd":
        dx, dw = api.linear_logprob_bwd(s["x"], s["w"], s["row_ptr"], s["row_sem"], s["target"], s["lse"],
                                        s["dlogp"])
        return {"dx": dx, "dw": dw}
    if op == "norm_fwd":
        y, h, rstd = api.rmsnorm_fwd(s["x"], s["weight"], s["res"], eps=s["eps"], mx8=s["mx8"])
        if s["mx8"]:
            q, scale = y
            C, D = q.shape
            y = (q.to(torch.bfloat16).view(C, D // BLOCK, BLOCK) * scale.to(torch.bfloat16)[:, :, None]).view(C, D)
        return {"y": y, "h": h, "rstd": rstd}
    if op == "norm_bwd":
        dx, dweight = api.rmsnorm_bwd(s["dy"], s["h"], s["weight"], s["rstd"], s["dh"])
        return {"dx": dx, "dweight": dweight}
    norm = s["set"].clip(s["max_norm"])
    return {"norm": norm, "out": s["out"]}


def _lse(z):
    m = z.amax(1, keepdim=True)
    return (m + torch.log(torch.exp(z - m).sum(1, keepdim=True)))[:, 0]


def _run_plain(s):
    op = s["op"]
    if op == "head_fwd":
        z = s["x"].float() @ s["w"].float().t()
        lse = _lse(z)
        y = s["target"].long()
        logp = z[s["sem_row"], y.clamp(min=0)] - lse[s["sem_row"]]
        return {"logp": torch.where(y >= 0, logp, torch.zeros_like(logp)), "lse": lse}
    if op == "head_bwd":
        x, w = s["x"].float(), s["w"].float()
        y = s["target"].long()
        g = torch.where(y >= 0, s["dlogp"], torch.zeros_like(s["dlogp"]))
        total = torch.zeros(x.shape[0], dtype=torch.float64, device=x.device).index_add_(0, s["sem_row"], g.double())
        dz = torch.exp(x @ w.t() - s["lse"][:, None]) * -total.float()[:, None]
        dz.index_put_((s["sem_row"], y.clamp(min=0)), g, accumulate=True)
        return {"dx": (dz @ w).to(s["x"].dtype), "dw": (dz.t() @ x).to(s["w"].dtype)}
    if op == "norm_fwd":
        h = s["x"].float() if s["res"] is None else s["x"].float() + s["res"].float()
        rstd = torch.rsqrt(h.square().mean(1) + s["eps"])
        y = h * rstd[:, None] * s["weight"]
        if s["mx8"]:
            C, D = y.shape
            b = y.view(C, D // BLOCK, BLOCK)
            m, e = torch.frexp(b.abs().amax(2, keepdim=True))
            e = torch.where(m > 0.875, e - 8, e - 9).clamp(-127, 127)    # 448 = 0.875 * 2^9 is e4m3's largest
            q = torch.ldexp(b, -e).to(torch.float8_e4m3fn)
            y = torch.ldexp(q.float(), e).view(C, D)
            return {"y": y.to(torch.bfloat16), "h": s["x"] if s["res"] is None else h.to(s["x"].dtype), "rstd": rstd}
        return {"y": y.to(s["x"].dtype), "h": s["x"] if s["res"] is None else h.to(s["x"].dtype), "rstd": rstd}
    if op == "norm_bwd":
        dy, h, r = s["dy"].float(), s["h"].float(), s["rstd"][:, None]
        n = h * r
        t = dy * s["weight"]
        dx = r * (t - n * (t * n).mean(1, keepdim=True))
        if s["dh"] is not None:
            dx = dx + s["dh"].float()
        return {"dx": dx.to(s["h"].dtype), "dweight": (dy * n).sum(0, dtype=torch.float64).float()}
    norm = torch.stack([t.float().square().sum(dtype=torch.float64) for t in s["grads"]]).sum().sqrt()
    coef = torch.where(norm > s["max_norm"], s["max_norm"] / norm, torch.ones_like(norm)).float()
    return {"norm": norm.float(), "out": [(t.float() * coef).to(t.dtype) for t in s["grads"]]}


# ---- what a pass cannot do without ----------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("head_fwd", "head_bwd"):
        C, V, D = case["rows"], case["vocab"], case["dim"]
        S = _positions(C)
        once = 2 * D * (C + V)
        if op == "head_fwd":
            return {"bytes": once + 4 * (C + 1) + 12 * S + 4 * C, "flops": 2 * C * V * D}
        return {"bytes": 2 * once + 4 * (C + 1) + 12 * S + 4 * C, "flops": 6 * C * V * D}
    if op in ("norm_fwd", "norm_bwd"):
        n, size = case["rows"] * case["dim"], 2 if case["dtype"] == "bf16" else 4
        if op == "norm_bwd":
            return {"bytes": n * size * (4 if case["residual"] else 3) + 8 * case["dim"] + 4 * case["rows"],
                    "flops": 12 * n}
        out = 1 + 1 / BLOCK if case["mx8"] else size
        return {"bytes": n * (size * (3 if case["residual"] else 2) + out) + 4 * case["dim"] + 4 * case["rows"],
                "flops": 6 * n}
    size = {"bf16": 2, "fp32": 4, "mixed": 3}[case["dtype"]]
    return {"bytes": 2 * size * case["values"], "flops": 3 * case["values"]}


# ---- the definitions in 64 bits -------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op in ("head_fwd", "head_bwd"):
        w = s["w"].double()
        C, S = s["x"].shape[0], s["target"].numel()
        logp = torch.zeros(S, dtype=torch.float64, device="cuda")
        lse = torch.empty(C, dtype=torch.float64, device="cuda")
        dx = torch.empty((C, w.shape[1]), dtype=torch.float64, device="cuda")
        dw = torch.zeros_like(w) if op == "head_bwd" else None
        ptr, sem = s["row_ptr"].long(), s["row_sem"].long()
        for a in range(0, C, 1024):
            b = min(C, a + 1024)
            xs = s["x"][a:b].double()
            z = torch.matmul(xs, w.T)
            pos = sem[ptr[a]:ptr[b]]
            row = torch.repeat_interleave(torch.arange(b - a, device="cuda"), ptr[a + 1:b + 1] - ptr[a:b])
            label = s["target"][pos].long()
            pos, row, label = pos[label >= 0], row[label >= 0], label[label >= 0]
            lse[a:b] = torch.logsumexp(z, 1)
            if op == "head_fwd":
                logp[pos] = torch.log_softmax(z, 1)[row, label]
                continue
            # lse is an input here: the softmax of the forward pass as it was handed over
            gs = s["dlogp"][pos].double()
            z = torch.exp(z - s["lse"][a:b].double()[:, None])
            tot = torch.zeros(b - a, dtype=torch.float64, device="cuda")
            tot.index_add_(0, row, gs)
            z.mul_(-tot[:, None])
            z.index_put_((row, label), gs, accumulate=True)
            dx[a:b] = torch.matmul(z, w)
            dw.addmm_(z.T, xs)
        return {"logp": logp, "lse": lse} if op == "head_fwd" else {"dx": dx, "dw": dw}
    if op == "norm_fwd":
        h = s["x"].double()
        if s["res"] is not None:
            h = h + s["res"].double()
        rstd = (h.pow(2).sum(1) / h.shape[1] + s["eps"]).pow(-0.5)
        y = h * rstd.unsqueeze(1) * s["weight"].double()
        if s["mx8"]:                    # the smallest power of two that keeps a block within 448, 4 significant bits
            b = y.unflatten(1, (-1, BLOCK))
            unit = torch.exp2(torch.ceil(torch.log2(b.abs().amax(2, keepdim=True) / 448)).clamp(-127, 127))
            step = torch.exp2(torch.floor(torch.log2((b / unit).abs().clamp(min=2.0 ** -6))) - 3)
            y = (torch.round(b / unit / step) * step * unit).flatten(1)
        return {"y": y, "h": h, "rstd": rstd}
    if op == "norm_bwd":
        dy, h, r, w = s["dy"].double(), s["h"].double(), s["rstd"].double().unsqueeze(1), s["weight"].double()
        inner = (dy * w * h).sum(1, keepdim=True) / h.shape[1]
        dx = dy * w * r - h * r.pow(3) * inner
        if s["dh"] is not None:
            dx = dx + s["dh"].double()
        return {"dx": dx, "dweight": (dy * h * r).sum(0)}
    norm = sum((t.double() ** 2).sum() for t in s["grads"]) ** 0.5
    coef = min(1.0, s["max_norm"] / float(norm))
    return {"norm": norm, "out": [t.double() * coef for t in s["grads"]]}
