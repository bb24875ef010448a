"""The update-tail example: its gradients against the fp64 oracle's chain, and its loss over
a few clipped steps.

Bounds.  The rows are rounded to bf16 twice on the way down (norm's output, the head's dx) and
once at the end, dz once; each is off by at most 2^-8 of its value, so a gradient that is a sum
of many such terms of either sign is off by less than 4 * 2^-8 = 1.6e-2 in relative L2."""
import os
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import tail as otail
from tests._parity import rel_l2

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from prefix_shared_chunkwise_gb300 import build
    build.build()


def test_gradients_against_the_oracle():
    from update_tail import Tail
    t = Tail("fig1_fp32", 256, 1003, seed=3)
    loss = t.gradients()
    norm = t.grads.clip(0.01)
    torch.cuda.synchronize()
    assert int(t.error) == 0
    f64 = lambda a: a.double().cpu().numpy()
    bf = lambda a: f64(a.to(torch.bfloat16))
    C, S = t.hidden.shape[0], t.target.numel()
    ptr, sem = t.row_ptr.cpu().numpy(), t.row_sem.cpu().numpy()
    sem_row = np.empty(S, np.int64)
    sem_row[sem] = np.repeat(np.arange(C), np.diff(ptr))
    y, h, rstd = otail.rmsnorm_fwd(bf(t.hidden), f64(t.residual), f64(t.norm_w), 1e-6)
    target, g = t.target.cpu().numpy().astype(np.int64), -f64(t.adv) / S
    logp, _ = otail.linear_logprob_fwd(y, bf(t.head), sem_row, target)
    assert abs(float(loss) + float((f64(t.adv) * logp).mean())) <= 2.0 ** -8 * abs(float(loss))
    dx, dhead = otail.linear_logprob_bwd(y, bf(t.head), sem_row, target, g)
    dh, dnorm = otail.rmsnorm_bwd(dx, h, f64(t.norm_w), rstd)
    for got, ref in ((t.d_hidden, dh), (t.d_head, dhead), (t.d_norm, dnorm)):
        assert rel_l2(f64(got), ref) <= 1.6e-2
    n, clipped = otail.grad_clip([dh, dhead, dnorm], 0.01)
    assert abs(float(norm) - n) <= 1.6e-2 * n
    for got, ref in zip(t.clipped, clipped):
        assert rel_l2(f64(got), ref) <= 3.2e-2


def test_loss_goes_down():
    from update_tail import main
    losses = main(["--steps", "12", "--dim", "264", "--vocab", "777"])
    assert losses[-1] < losses[0] and all(np.isfinite(losses))


def test_buffers_of_a_call_belong_to_its_stream():
    """Calls on a second stream that is still busy, their workspaces dropped at once: what the
    current stream then allocates and fills must not reach them.  Same kernels in the same order
    of sums: results are equal to the bit."""
    from prefix_shared_chunkwise_gb300.api import GradSet, linear_logprob_bwd, linear_logprob_fwd, rmsnorm_bwd, rmsnorm_fwd
    gen = torch.Generator().manual_seed(5)
    rnd = lambda *shape: torch.randn(*shape, generator=gen)
    C, V, D = 200, 1500, 136
    x, w = rnd(C, D).bfloat16().cuda(), (0.1 * rnd(V, D)).bfloat16().cuda()
    ptr = torch.arange(C + 1, dtype=torch.int32).cuda()
    sem = torch.randperm(C, generator=gen).int().cuda()
    target, dlogp = torch.randint(0, V, (C,), generator=gen).int().cuda(), rnd(C).cuda()
    weight, dy = rnd(D).cuda(), rnd(C, D).bfloat16().cuda()
    grads = [rnd(70001).cuda(), rnd(513).bfloat16().cuda()]

    def calls(stream):
        clipped = [torch.zeros_like(g) for g in grads]
        torch.cuda.synchronize()
        if stream is not None:
            with torch.cuda.stream(stream):
                torch.cuda._sleep(20_000_000)
        logp, lse = linear_logprob_fwd(x, w, ptr, sem, target, stream=stream)
        dx, dw = linear_logprob_bwd(x, w, ptr, sem, target, lse, dlogp, stream=stream)
        y, h, rstd = rmsnorm_fwd(x, weight, dy, stream=stream)
        dn, dweight = rmsnorm_bwd(dy, h, weight, rstd, stream=stream)
        norm = GradSet(grads, clipped).clip(0.5, stream=stream)
        junk = [torch.full((n,), 0x7f, dtype=torch.uint8, device="cuda")
                for n in (256, 4096, 1 << 16, 1 << 18, 1 << 20, 1 << 22) for _ in range(8)]
        torch.cuda.synchronize()
        del junk
        return [logp, lse, dx, dw, y, h, rstd, dn, dweight, norm, *clipped]

    here = calls(None)
    there = calls(torch.cuda.Stream())
    for a, b in zip(here, there):
        assert torch.equal(a, b)


def test_every_entry_point_asks_for_the_current_device(monkeypatch):
    """With another device current (by its name only: one GPU is enough) no entry point launches."""
    from prefix_shared_chunkwise_gb300 import api
    bf = dict(dtype=torch.bfloat16, device="cuda")
    x, w, i = torch.zeros(4, 64, **bf), torch.zeros(64, device="cuda"), torch.zeros(5, dtype=torch.int32, device="cuda")
    head, f4, f5 = torch.zeros(10, 64, **bf), torch.zeros(4, device="cuda"), torch.zeros(5, device="cuda")
    q = torch.zeros(4, 1, 128, **bf)
    pl = api.Plan(np.array([-1], np.int32), np.array([4], np.int64), 64).upload()
    grads = api.GradSet([w])
    calls = [lambda: api.rmsnorm_fwd(x, w), lambda: api.rmsnorm_bwd(x, x, w, f4), lambda: grads.norm(),
             lambda: grads.clip(1.0), lambda: api.GradSet([w]), lambda: api.linear_logprob_fwd(x, head, i, i, i),
             lambda: api.linear_logprob_bwd(x, head, i, i, i, f4, f5), lambda: api.logprob_fwd(x, i, i, i),
             lambda: api.logprob_bwd(x, i, i, i, f4, f5), lambda: api.attn_fwd(pl, q, q, q),
             lambda: api.attn_bwd(pl, q, q, q, q, f4.view(4, 1), q),
             lambda: api.conv_fwd(pl, x, torch.zeros(64, 4, device="cuda")),
             lambda: api.conv_bwd(pl, x, torch.zeros(64, 4, device="cuda"), None, x),
             lambda: api.kda_fwd(pl, q, q, q, q, q[:, :, 0].contiguous()), lambda: pl.device_error(), lambda: pl.upload()]
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for call in calls:
        with pytest.raises(ValueError, match="current device is cuda:1"):
            call()


def test_a_wait_that_ran_out_is_not_lost_without_an_error_word():
    """Calls that are given no error word report in the library's own, which says so once."""
    from prefix_shared_chunkwise_gb300 import _lib, api
    assert api.device_error() == 0
    assert _lib.lib().harts_selftest_timeout(None, 2_000_000, torch.cuda.current_stream().cuda_stream) == 0
    assert api.device_error() == 3 and api.device_error() == 0
    gen = torch.Generator().manual_seed(6)
    x, w = torch.randn(70, 256, generator=gen).bfloat16().cuda(), torch.randn(500, 256, generator=gen).bfloat16().cuda()
    ptr = torch.arange(71, dtype=torch.int32).cuda()
    logp, lse = api.linear_logprob_fwd(x, w, ptr, ptr[:70].clone(), ptr[:70].clone())
    api.linear_logprob_bwd(x, w, ptr, ptr[:70].clone(), ptr[:70].clone(), lse, logp)
    y, h, rstd = api.rmsnorm_fwd(x, torch.ones(256, device="cuda"))
    api.rmsnorm_bwd(y, h, torch.ones(256, device="cuda"), rstd)
    assert api.device_error() == 0 and torch.isfinite(lse).all()


FIRST_CALL = """
import sys, torch
from prefix_shared_chunkwise_gb300.api import device_error, linear_logprob_bwd, linear_logprob_fwd
gen = torch.Generator().manual_seed(7)
x, w = torch.randn(70, 72, generator=gen).bfloat16().cuda(), torch.randn(500, 72, generator=gen).bfloat16().cuda()
ptr = torch.arange(71, dtype=torch.int32).cuda()
sem, tgt, g = ptr[:70].clone(), ptr[:70].clone(), torch.randn(70, generator=gen).cuda()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    logp, lse = linear_logprob_fwd(x, w, ptr, sem, tgt)
    dx, dw = linear_logprob_bwd(x, w, ptr, sem, tgt, lse, g)
graph.replay()
torch.cuda.synchronize()
logp2, lse2 = linear_logprob_fwd(x, w, ptr, sem, tgt)
dx2, dw2 = linear_logprob_bwd(x, w, ptr, sem, tgt, lse2, g)
same = [torch.equal(a, b) for a, b in ((logp, logp2), (lse, lse2), (dx, dx2), (dw, dw2))]
sys.exit(0 if all(same) and device_error() == 0 else 1)
"""


def test_the_first_call_of_a_process_may_be_captured():
    """What a first call looks up (the error word, a kernel's shared memory) it finds in a capture."""
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
