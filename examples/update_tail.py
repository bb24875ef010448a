"""The tail of one policy update over a rollout tree, with its gradients.

    python examples/update_tail.py [--workload fig1_fp32] [--dim 512] [--vocab 5000] [--steps 30]

Hidden rows of the compact layout (random here; a model's last layer in earnest) go through
the residual's addition and the final norm, the vocabulary projection with per-position
log-probabilities, a policy loss  -sum_s A_s logp[s] / S  over all trajectories of the tree,
back through both, and a clipped gradient step on the norm's weight, the vocabulary weight and
the rows.  No C x V array is formed at any point."""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

from prefix_shared_chunkwise_gb300.api import (GradSet, Plan, linear_logprob_bwd, linear_logprob_fwd, rmsnorm_bwd,
                                               rmsnorm_fwd, semantic_map)
from prefix_shared_chunkwise_gb300.synth import make_tree


class Tail:
    """Parameters (fp32 masters, bf16 copies for the kernels), buffers and the tree's map."""

    def __init__(self, workload, dim, vocab, seed=0, device="cuda"):
        parent, seg_len = make_tree(workload)
        plan = Plan(parent, seg_len, 64)
        _, row_ptr, row_sem = semantic_map(plan)
        self.row_ptr, self.row_sem = (torch.as_tensor(a, device=device) for a in (row_ptr, row_sem))
        C, S = plan.info["C"], len(row_sem)
        g = torch.Generator(device=device).manual_seed(seed)
        rand = lambda *shape: torch.randn(shape, generator=g, device=device)
        self.hidden = rand(C, dim)                          # the last layer's output
        self.residual = rand(C, dim).to(torch.bfloat16)     # the stream it is added to
        self.norm_w = torch.ones(dim, device=device)
        self.head = rand(vocab, dim) / dim ** 0.5
        self.target = torch.randint(0, vocab, (S,), generator=g, device=device, dtype=torch.int32)
        self.adv = torch.rand(S, generator=g, device=device)
        self.error = torch.zeros(1, dtype=torch.int32, device=device)
        bf = torch.bfloat16
        self.d_hidden = torch.empty((C, dim), dtype=bf, device=device)
        self.d_head = torch.empty((vocab, dim), dtype=bf, device=device)
        self.d_norm = torch.empty(dim, device=device)
        self.clipped = [torch.empty(t.shape, device=device) for t in (self.d_hidden, self.d_head, self.d_norm)]
        self.grads = GradSet([self.d_hidden, self.d_head, self.d_norm], self.clipped)

    def gradients(self):
        """One forward and backward pass; returns the loss.  Leaves d_hidden, d_head, d_norm."""
        S, head = self.target.numel(), self.head.to(torch.bfloat16)
        x, h, rstd = rmsnorm_fwd(self.hidden.to(torch.bfloat16), self.norm_w, self.residual)
        logp, lse = linear_logprob_fwd(x, head, self.row_ptr, self.row_sem, self.target, error=self.error)
        loss = -(self.adv * logp).mean()
        dx, _ = linear_logprob_bwd(x, head, self.row_ptr, self.row_sem, self.target, lse, -self.adv / S,
                                   dweight=self.d_head, error=self.error)
        rmsnorm_bwd(dx, h, self.norm_w, rstd, dx=self.d_hidden, dweight=self.d_norm, error=self.error)
        return loss

    def step(self, lr, max_norm):
        """gradients(), clipped to max_norm, and one step down them; returns (loss, norm)."""
        loss = self.gradients()
        norm = self.grads.clip(max_norm)
        for p, d in zip((self.hidden, self.head, self.norm_w), self.clipped):
            p.add_(d, alpha=-lr)
        return loss, norm


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--workload", default="fig1_fp32", help="a forest of synth.WORKLOADS")
    ap.add_argument("--dim", type=int, default=512)
    ap.add_argument("--vocab", type=int, default=5000)
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--lr", type=float, default=40.0)
    ap.add_argument("--max-norm", type=float, default=0.05)
    a = ap.parse_args(argv)
    tail = Tail(a.workload, a.dim, a.vocab)
    losses = []
    for i in range(a.steps):
        loss, norm = tail.step(a.lr, a.max_norm)
        losses.append(float(loss))
        if i % 10 == 0 or i == a.steps - 1:
            print(f"step {i:3d}  loss {losses[-1]:.4f}  gradient norm {float(norm):.4f}")
    if int(tail.error) != 0:
        raise RuntimeError("a bounded device wait ran out")
    return losses


if __name__ == "__main__":
    main()
