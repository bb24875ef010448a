"""One recurrent block over a rollout tree, forward and backward.

    python examples/recurrent_block.py [--workload fig1_fp32] [--dim 512] [--heads 4] [--steps 20]

The block's input is the normed residual stream.  Three projections give the recurrence's input,
its gate and the output's gate; the input goes through the short convolution and the gated
recurrence over the tree, every head's output is normed and gated, a projection brings it back, and
one pass norms it, adds it to the stream and norms the stream for the next block.  Each of these runs once per
compact row.  The loss is a fixed linear function of the block's two outputs, so that the gradients of
all parameters can be looked at."""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

from prefix_shared_chunkwise_gb300.api import (Plan, block_norm_bwd, block_norm_fwd, conv_bwd, conv_fwd, linear_bwd,
                                               linear_fwd, scan_bwd, scan_fwd)
from prefix_shared_chunkwise_gb300.synth import make_tree


class RecurrentBlock:
    """Parameters: fp32 vectors, bf16 matrices.  forward() keeps what backward() reads."""

    def __init__(self, dim, heads, head_dim=128, width=4, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        rand = lambda *shape: torch.randn(shape, generator=g, device=device)
        inner = heads * head_dim
        self.heads, self.head_dim, self.scale = heads, head_dim, 0.5
        matrix = lambda n, k: (rand(n, k) / k ** 0.5).bfloat16()
        self.p = {"w_in": matrix(inner, dim), "w_decay": matrix(inner, dim), "b_decay": 1 + rand(inner), "w_gate": matrix(inner, dim),
                  "w_out": matrix(dim, inner), "conv": 0.4 * rand(inner, width), "head": 1 + 0.1 * rand(head_dim),
                  "post": 1 + 0.1 * rand(dim), "pre": 1 + 0.1 * rand(dim)}

    def forward(self, plan, n, stream):
        """n, stream: [C, dim] bf16.  Returns (the stream behind the block, its norm for the next one)."""
        p, rows = self.p, (-1, self.head_dim)
        x, _ = linear_fwd(n, p["w_in"])
        c = conv_fwd(plan, x, p["conv"], activation="silu")
        t, _ = linear_fwd(n, p["w_decay"], p["b_decay"])
        decay = torch.nn.functional.logsigmoid(t.float()).bfloat16()        # e^decay = sigmoid(t)
        h = scan_fwd(plan, c, decay, form="mix")
        gate, _ = linear_fwd(n, p["w_gate"])
        o, _, r_head, _ = block_norm_fwd(h.view(rows), post_weight=p["head"], gate=gate.view(rows), gate_act="silu")
        y, _ = linear_fwd(o.view(h.shape), p["w_out"])
        s, m, r_post, r_pre = block_norm_fwd(y, post_weight=p["post"], residual=stream, scale=self.scale, pre_weight=p["pre"])
        self.kept = dict(plan=plan, n=n, x=x, c=c, t=t, decay=decay, h=h, gate=gate, o=o.view(h.shape), r_head=r_head, y=y, s=s,
                         r_post=r_post, r_pre=r_pre)
        return s, m

    def backward(self, d_s, d_m):
        """Gradients of forward()'s two outputs to (d_n, d_stream, dict of the parameters')."""
        k, p, rows, d = self.kept, self.p, (-1, self.head_dim), {}
        b = block_norm_bwd(k["y"], k["s"], d_m, d_s, post_weight=p["post"], scale=self.scale, pre_weight=p["pre"],
                           rstd_post=k["r_post"], rstd_pre=k["r_pre"])
        d["post"], d["pre"] = b["dpost_weight"], b["dpre_weight"]
        d_o, d["w_out"], _ = linear_bwd(k["o"], p["w_out"], b["dy"])
        hb = block_norm_bwd(k["h"].view(rows), None, None, d_o.view(rows), post_weight=p["head"], gate=k["gate"].view(rows),
                            gate_act="silu", rstd_post=k["r_head"])
        d["head"] = hb["dpost_weight"]
        shape = k["h"].shape
        d_c, d_decay = scan_bwd(k["plan"], k["c"], k["decay"], k["h"], hb["dy"].view(shape), form="mix")
        d_t = (d_decay.float() * torch.sigmoid(-k["t"].float())).bfloat16()
        d_x, d["conv"], _ = conv_bwd(k["plan"], k["x"], p["conv"], None, d_c, activation="silu")
        dn1, d["w_in"], _ = linear_bwd(k["n"], p["w_in"], d_x)
        dn2, d["w_decay"], d["b_decay"] = linear_bwd(k["n"], p["w_decay"], d_t, with_bias=True)
        dn3, d["w_gate"], _ = linear_bwd(k["n"], p["w_gate"], hb["dgate"].view(shape))
        return dn1.float() + dn2.float() + dn3.float(), b["dresidual"], d


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--workload", default="fig1_fp32", help="a forest of synth.WORKLOADS")
    ap.add_argument("--dim", type=int, default=512)
    ap.add_argument("--heads", type=int, default=4)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args(argv)
    parent, seg_len = make_tree(a.workload)
    plan = Plan(parent, seg_len, 64).upload()
    C = plan.info["C"]
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda: torch.randn((C, a.dim), generator=g, device="cuda").bfloat16()
    n, stream, d_s, d_m = rand(), rand(), rand(), rand()
    block = RecurrentBlock(a.dim, a.heads)
    block.forward(plan, n, stream)
    block.backward(d_s, d_m)
    torch.cuda.synchronize()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(a.steps):
        s, m = block.forward(plan, n, stream)
        d_n, d_stream, grads = block.backward(d_s, d_m)
    end.record()
    torch.cuda.synchronize()
    if plan.device_error() != 0:
        raise RuntimeError("a bounded device wait ran out")
    print(f"{C} compact rows, {a.dim} channels, {a.heads} heads: {start.elapsed_time(end) / a.steps:.3f} ms a step")
    for name, t in grads.items():
        print(f"  d {name:8s} {tuple(t.shape)}  norm {float(t.float().norm()):.4g}")
    return grads


if __name__ == "__main__":
    main()
