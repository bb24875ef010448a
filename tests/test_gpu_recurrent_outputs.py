"""harts_linear_bwd and harts_block_norm_bwd through the C interface with some of the outputs left out: those that
are asked for keep their bits, and nothing else is written."""
import ctypes
import itertools

import pytest

torch = pytest.importorskip("torch")

from prefix_shared_chunkwise_gb300 import _lib as L
from prefix_shared_chunkwise_gb300.api import block_norm_bwd, block_norm_fwd, linear_bwd, linear_fwd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from prefix_shared_chunkwise_gb300 import build
    build.build()


def _at(t):
    return None if t is None else t.data_ptr()


@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("C,K,N", [(2, 264, 136), (300, 1032, 520), (2500, 264, 72)])
def test_linear_bwd(C, K, N, act):
    g = torch.Generator(device="cuda").manual_seed(C)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    x, w, dy = rand(C, K), rand(N, K), rand(C, N)
    z = linear_fwd(x, w, activation=act, keep_z=True)[1]
    want = linear_bwd(x, w, dy, z, activation=act, with_bias=True)
    lib, code = L.lib(), {"none": L.HARTS_ACT_NONE, "gelu": L.HARTS_ACT_GELU}[act]
    for asked in itertools.product((False, True), repeat=3):
        if not any(asked):
            continue
        out = [torch.full_like(t, 7.0) if on else None for t, on in zip(want, asked)]
        nb = lib.harts_linear_bwd_workspace_bytes(C, K, N, code, asked[2])
        ws = torch.full((max(nb, 1) + 256,), 0xff, dtype=torch.uint8, device="cuda")
        f = L.LinearArgs(C, K, N, L.HARTS_BF16, code, _at(x), _at(w), None, None, None, _at(z), None, _at(ws) if nb else None, nb)
        a = L.LinearBwdArgs(f, _at(dy), *map(_at, out))
        L.check(lib.harts_linear_bwd(ctypes.byref(a), torch.cuda.current_stream().cuda_stream), "harts_linear_bwd")
        torch.cuda.synchronize()
        assert all(o is None or torch.equal(o, t) for o, t in zip(out, want)), asked
        assert bool((ws[nb:] == 0xff).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("C,D", [(700, 264), (40, 5001), (300, 131)])
def test_block_norm_bwd(C, D, dtype):
    g = torch.Generator(device="cuda").manual_seed(C)
    rand = lambda: torch.randn((C, D), generator=g, device="cuda").to(dtype)
    y, gate, res, dn, dh = rand(), rand(), rand(), rand(), rand()
    w = torch.rand(D, generator=g, device="cuda") + 0.5
    kw = dict(post_weight=w, gate=gate, scale=0.5, pre_weight=w)
    h, _, r1, r2 = block_norm_fwd(y, residual=res, **kw)
    want = block_norm_bwd(y, h, dn, dh, rstd_post=r1, rstd_pre=r2, **kw)
    lib, code = L.lib(), L.HARTS_BF16 if dtype == torch.bfloat16 else L.HARTS_FP32
    nb = lib.harts_block_norm_bwd_workspace_bytes(C, D, code)
    for with_res, with_gate in itertools.product((False, True), repeat=2):
        ws = torch.full((nb + 256,), 0xff, dtype=torch.uint8, device="cuda")
        out = {k: torch.full_like(v, 7.0) for k, v in want.items()}
        f = L.BlockNormArgs(C, D, code, L.HARTS_GATE_SILU, 0.5, 0.0, _at(y), _at(gate), None, _at(w), _at(w), _at(h), None, _at(r1), _at(r2), None)
        a = L.BlockNormBwdArgs(f, _at(dn), _at(dh), _at(out["dy"]), _at(out["dresidual"]) if with_res else None,
                               _at(out["dgate"]) if with_gate else None, _at(out["dpost_weight"]), _at(out["dpre_weight"]), _at(ws), nb)
        L.check(lib.harts_block_norm_bwd(ctypes.byref(a), torch.cuda.current_stream().cuda_stream), "harts_block_norm_bwd")
        torch.cuda.synchronize()
        for k, v in want.items():
            left = (k == "dresidual" and not with_res) or (k == "dgate" and not with_gate)
            assert bool((out[k] == 7.0).all()) if left else torch.equal(out[k], v), k
        assert bool((ws[nb:] == 0xff).all())
