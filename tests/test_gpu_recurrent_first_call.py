"""A process whose first call of an operator is captured into a graph: nothing that a call sets up once (shared memory's
limit, occupancy, the library's error word, tensor maps) may need a call outside a capture."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

PROGRAM = """
import torch
from prefix_shared_chunkwise_gb300.api import (Plan, block_norm_bwd, block_norm_fwd, device_error, linear_bwd, linear_fwd, scan_bwd,
                                               scan_fwd)
C, D = 300, 264
plan = Plan([-1, 0, 0], [100, 150, 50], 64).upload()
x, w = torch.randn(C, D, device="cuda").bfloat16(), torch.randn(D, D, device="cuda").bfloat16() / 16
g, n = -torch.rand(C, D, device="cuda").bfloat16(), torch.rand(D, device="cuda") + 0.5
torch.cuda.synchronize()

def run():
    y, z = linear_fwd(x, w, n, activation="silu", keep_z=True)
    h = scan_fwd(plan, y, g, form="mix")
    kw = dict(post_weight=n, gate=x, pre_weight=n)
    s, m, r1, r2 = block_norm_fwd(h, residual=y, **kw)
    d = block_norm_bwd(h, s, m, s, rstd_post=r1, rstd_pre=r2, **kw)
    dy, dg = scan_bwd(plan, y, g, h, d["dy"], form="mix")
    return [y, z, h, s, m, dy, dg, d["dpost_weight"], d["dpre_weight"], *linear_bwd(x, w, dy, z, activation="silu", with_bias=True)]

graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = run()
for t in got:
    t.zero_()
graph.replay()
want = run()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want))
assert plan.device_error() == 0 and device_error() == 0
"""


def test_captured_first():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from prefix_shared_chunkwise_gb300 import build
    build.build()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
