"""scan, block_norm and linear in the order in which a recurrent block uses them, with the short
convolution between them (examples/recurrent_block.py): outputs and all gradients against torch's
autograd of the same formulas in 64 bits on the CPU.

Bound.  Every tensor between two operators is rounded to bf16: half a step is at most 2^-8 of a value,
and in relative L2 over many values 2^-8 / sqrt 3 at most, 2.3e-3.  On the longest way, from an output's gradient
through y, o, h, decay, t and back, there are at most eight of them forward and eight
backward; every operator here passes on relative errors of its input about unchanged (norms and
projections by random matrices keep lengths): 16 x 2.3e-3 = 3.6e-2 if they all added up."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from prefix_shared_chunkwise_gb300 import build
    build.build()


def _before(plan, parent, seg_len):
    """Row before each compact row on its trajectory, -1 at a root's start."""
    off = plan.arrays()["seg_offset"]
    out = np.arange(plan.info["C"]) - 1
    for v, p in enumerate(parent):
        out[off[v]] = -1 if p < 0 else off[p] + seg_len[p] - 1
    return out


def _norm(x, w):
    return x / torch.sqrt((x * x).mean(1, keepdim=True) + 1e-6) * w


def _reference(block, before, n, stream, d_s, d_m):
    p = {k: v.detach().double().cpu().requires_grad_() for k, v in block.p.items()}
    n, stream = (t.detach().double().cpu().requires_grad_() for t in (n, stream))
    x = n @ p["w_in"].T
    width, C = p["conv"].shape[1], len(x)
    taps, at = [], torch.arange(C)
    zero = torch.zeros(1, x.shape[1], dtype=torch.float64)
    padded = torch.cat([x, zero])
    for j in range(width):
        taps.append(padded[at] * p["conv"][:, width - 1 - j])
        at = torch.tensor([before[i] if 0 <= i < C and before[i] >= 0 else C for i in at.tolist()])
    c = sum(taps)
    c = c * torch.sigmoid(c)
    a = torch.sigmoid(n @ p["w_decay"].T + p["b_decay"])
    rows = [None] * C
    for r in range(C):                                      # a row's parent has a lower number
        b = (1 - a[r]) * c[r]
        rows[r] = b if before[r] < 0 else a[r] * rows[before[r]] + b
    h = torch.stack(rows)
    gate = n @ p["w_gate"].T
    o = (_norm(h.reshape(-1, block.head_dim), p["head"])).reshape(h.shape) * gate * torch.sigmoid(gate)
    s = stream + block.scale * _norm(o @ p["w_out"].T, p["post"])
    m = _norm(s, p["pre"])
    (s * d_s.double().cpu()).sum().add((m * d_m.double().cpu()).sum()).backward()
    return s.detach(), m.detach(), n.grad, stream.grad, {k: v.grad for k, v in p.items()}


def _rel(a, b):
    a, b = a.double().cpu(), b.double()
    return float((a - b).norm() / b.norm())


@pytest.mark.parametrize("forest", [([-1, 0, 0, 1, 1, -1, 5], [70, 30, 9, 1, 20, 140, 3]), ([-1], [200])])
def test_block_against_autograd(forest):
    from examples.recurrent_block import RecurrentBlock
    from prefix_shared_chunkwise_gb300.api import Plan
    parent, seg_len = forest
    plan = Plan(parent, seg_len, 64).upload()
    C, dim = plan.info["C"], 264
    g = torch.Generator(device="cuda").manual_seed(5)
    rand = lambda: torch.randn((C, dim), generator=g, device="cuda").bfloat16()
    n, stream, d_s, d_m = rand(), rand(), rand(), rand()
    block = RecurrentBlock(dim, 2)
    s, m = block.forward(plan, n, stream)
    d_n, d_stream, grads = block.backward(d_s, d_m)
    torch.cuda.synchronize()
    assert plan.device_error() == 0
    rs, rm, rn, rstream, rp = _reference(block, _before(plan, parent, seg_len), n, stream, d_s, d_m)
    bound = 16 * 2.0 ** -8 / 3 ** 0.5
    errors = {"s": _rel(s, rs), "m": _rel(m, rm), "n": _rel(d_n, rn), "stream": _rel(d_stream, rstream),
              **{k: _rel(grads[k], rp[k]) for k in rp}}
    assert max(errors.values()) <= bound, errors


def test_block_is_captured_as_a_whole():
    """One graph of a step, replayed on other inputs in the same buffers, equals the eager step to the bit."""
    from examples.recurrent_block import RecurrentBlock
    from prefix_shared_chunkwise_gb300.api import Plan
    plan = Plan([-1, 0, 0, -1], [300, 40, 77, 130], 64).upload()
    C, dim = plan.info["C"], 256
    g = torch.Generator(device="cuda").manual_seed(6)
    rand = lambda: torch.randn((C, dim), generator=g, device="cuda").bfloat16()
    n, stream, d_s, d_m = rand(), rand(), rand(), rand()
    block = RecurrentBlock(dim, 2)

    def step():
        s, m = block.forward(plan, n, stream)
        d_n, d_stream, grads = block.backward(d_s, d_m)
        return [s, m, d_n, d_stream, *grads.values()]
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(2):
        for t in (n, stream, d_s, d_m):
            t.copy_(rand())
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert plan.device_error() == 0


def test_the_example_runs():
    from examples import recurrent_block
    grads = recurrent_block.main(["--steps", "2", "--dim", "128", "--heads", "1"])
    assert all(bool(t.isfinite().all()) and bool((t != 0).any()) for t in grads.values())
