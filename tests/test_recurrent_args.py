"""What the entry points around a recurrent layer (scan, block_norm, linear) refuse, on the host: every
case returns its error code before anything is enqueued, so none of them needs a GPU."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from prefix_shared_chunkwise_gb300 import _lib as L

P = 1 << 20          # well-aligned addresses that are never dereferenced
Q = [P * (i + 2) for i in range(12)]
EINVAL, EUNSUPPORTED, EOVERFLOW, ESMALLBUF, ENOPLAN = -1, -2, -3, -4, -8


@pytest.fixture(scope="module", autouse=True)
def built():
    from prefix_shared_chunkwise_gb300 import build
    build.build()


def _args(cls, base, **change):
    a = cls()
    for k, v in {**base, **change}.items():
        if "." in k:
            o, f = k.split(".")
            setattr(getattr(a, o), f, v)
        else:
            setattr(a, k, v)
    return a


def _fwd(base):
    return {f"fwd.{k}": v for k, v in base.items()}


@pytest.fixture(scope="module")
def plan():
    from prefix_shared_chunkwise_gb300.api import Plan
    return Plan([-1, 0, 0], [5, 6, 7], 64)


SCAN = dict(channels=64, dtype=1, form=0, x=Q[0], g=Q[1], h=Q[2], workspace=P, workspace_bytes=1 << 30)
SCAN_BWD = {**_fwd(SCAN), "d_h": Q[3], "dx": Q[4], "dg": Q[5]}
SCAN_BAD = [
    (EINVAL, dict(x=None)), (EINVAL, dict(g=None)), (EINVAL, dict(h=None)), (EINVAL, dict(x=P + 8)), (EINVAL, dict(g=P + 4)),
    (EINVAL, dict(h=P + 2)), (EINVAL, dict(h0=P + 4)), (EINVAL, dict(final_state=P + 8)), (EINVAL, dict(workspace=P + 8)),
    (EINVAL, dict(channels=0)), (EINVAL, dict(channels=60)), (EINVAL, dict(channels=-8)), (EINVAL, dict(form=2)),
    (EINVAL, dict(form=-1)), (EINVAL, dict(h0=P, final_state=P)), (EINVAL, dict(h=Q[0])), (EINVAL, dict(h=Q[1])), (EUNSUPPORTED, dict(dtype=2)),
    (EUNSUPPORTED, dict(dtype=-1)),
]


@pytest.mark.parametrize("rc,change", SCAN_BAD + [(ENOPLAN, {})])
def test_scan_fwd_refuses(plan, rc, change):
    assert L.lib().harts_scan_fwd(plan.handle, ctypes.byref(_args(L.ScanFwdArgs, SCAN, **change)), None) == rc
    assert L.lib().harts_last_error()


@pytest.mark.parametrize("rc,change", [(rc, _fwd(c)) for rc, c in SCAN_BAD] + [
    (EINVAL, dict(d_h=None)), (EINVAL, dict(dx=None)), (EINVAL, dict(dg=None)), (EINVAL, dict(d_h=P + 8)), (EINVAL, dict(dx=P + 2)),
    (EINVAL, dict(dg=P + 4)), (EINVAL, dict(d_final=P + 4)), (EINVAL, dict(dh0=P + 8)), (EINVAL, dict(dx=Q[0])),
    (EINVAL, dict(dg=Q[1])), (EINVAL, dict(dx=Q[2])), (EINVAL, dict(dg=Q[3])), (EINVAL, dict(dx=Q[5])), (EINVAL, dict(dh0=P, d_final=P)), (EINVAL, {"dh0": P, "fwd.h0": P}), (ENOPLAN, {}),
])
def test_scan_bwd_refuses(plan, rc, change):
    assert L.lib().harts_scan_bwd(plan.handle, ctypes.byref(_args(L.ScanBwdArgs, SCAN_BWD, **change)), None) == rc


def test_scan_sizes(plan):
    from prefix_shared_chunkwise_gb300.api import Plan
    lib = L.lib()
    assert lib.harts_scan_fwd(None, ctypes.byref(_args(L.ScanFwdArgs, SCAN)), None) == EINVAL
    assert lib.harts_scan_fwd(plan.handle, None, None) == EINVAL and lib.harts_scan_bwd(plan.handle, None, None) == EINVAL
    nb = lib.harts_scan_workspace_bytes
    assert nb(plan.handle, 64, 1) > 0 and nb(plan.handle, 64, 0) > 0
    assert nb(None, 64, 1) == nb(plan.handle, 60, 1) == nb(plan.handle, 0, 1) == nb(plan.handle, 64, 2) == 0
    # segments that do not follow one another need none
    assert nb(Plan([-1, -1], [128, 1], 64).handle, 64, 1) == 0
    assert nb(Plan([-1, -1], [129, 1], 64).handle, 64, 1) > 0


NORM = dict(C=4, D=64, dtype=1, gate_act=1, scale=1.0, eps=1e-6, y=Q[0], gate=Q[1], residual=Q[2], post_weight=Q[3],
            pre_weight=Q[4], h=Q[5], n=Q[6], rstd_post=P, rstd_pre=P)
NORM_BWD = {**_fwd(NORM), "d_n": Q[7], "d_h": Q[8], "dy": Q[9], "dresidual": Q[10], "dgate": Q[11], "dpost_weight": P,
            "dpre_weight": P, "workspace": P, "workspace_bytes": 1 << 30}
NORM_BAD = [
    (EINVAL, dict(y=None)), (EINVAL, dict(h=None)), (EINVAL, dict(post_weight=None, pre_weight=None, n=None)), (EINVAL, dict(y=P + 8)),
    (EINVAL, dict(gate=P + 2)), (EINVAL, dict(post_weight=P + 4)), (EINVAL, dict(pre_weight=P + 4)),
    (EINVAL, dict(h=P + 8)), (EINVAL, dict(C=-1)), (EINVAL, dict(D=0)), (EINVAL, dict(scale=float("inf"))),
    (EINVAL, dict(scale=float("nan"))), (EINVAL, dict(gate_act=3)), (EINVAL, dict(gate_act=-1)), (EUNSUPPORTED, dict(dtype=2)),
    (EUNSUPPORTED, dict(D=8193)),
]


@pytest.mark.parametrize("rc,change", NORM_BAD + [
    (EINVAL, dict(n=None)), (EINVAL, dict(pre_weight=None)), (EINVAL, dict(n=Q[5])), (EINVAL, dict(n=P + 2)), (EINVAL, dict(residual=P + 8)),
    (EINVAL, dict(eps=-1.0)), (EINVAL, dict(eps=float("nan"))), (EINVAL, dict(eps=float("inf"))),
])
def test_block_norm_fwd_refuses(rc, change):
    assert L.lib().harts_block_norm_fwd(ctypes.byref(_args(L.BlockNormArgs, NORM, **change)), None) == rc
    assert L.lib().harts_last_error()


@pytest.mark.parametrize("rc,change", [(rc, _fwd(c)) for rc, c in NORM_BAD] + [
    (EINVAL, {"fwd.rstd_post": None}), (EINVAL, {"fwd.rstd_pre": None}), (EINVAL, dict(d_n=None)), (EINVAL, dict(d_n=P + 2)),
    (EINVAL, dict(d_h=P + 8)), (EINVAL, dict(dy=None)), (EINVAL, dict(dy=P + 8)), (EINVAL, dict(dresidual=P + 2)), (EINVAL, dict(dgate=P + 4)),
    (EINVAL, dict(dpost_weight=None)), (EINVAL, dict(dpre_weight=None)), (EINVAL, {"fwd.gate": None}), (EINVAL, dict(dy=Q[10])),
    (EINVAL, dict(dy=Q[11])), (EINVAL, dict(dgate=Q[10])), (EINVAL, {"fwd.pre_weight": None, "d_h": None}),
    (ESMALLBUF, dict(workspace=None)), (ESMALLBUF, dict(workspace_bytes=8)), (EINVAL, dict(workspace=P + 8)),
])
def test_block_norm_bwd_refuses(rc, change):
    assert L.lib().harts_block_norm_bwd(ctypes.byref(_args(L.BlockNormBwdArgs, NORM_BWD, **change)), None) == rc


LINEAR = dict(C=300, K=64, N=72, dtype=1, activation=2, x=Q[0], weight=Q[1], bias=Q[2], residual=Q[3], y=Q[4], z=Q[5], workspace=P,
              workspace_bytes=1 << 30)
LINEAR_BWD = {**_fwd(LINEAR), "d_y": Q[6], "dx": Q[7], "dweight": Q[8], "dbias": Q[9]}
LINEAR_BAD = [
    (EINVAL, dict(x=None)), (EINVAL, dict(weight=None)), (EINVAL, dict(x=P + 8)), (EINVAL, dict(weight=P + 2)), (EINVAL, dict(z=P + 8)),
    (EINVAL, dict(C=-1)), (EINVAL, dict(K=0)), (EINVAL, dict(N=-8)), (EINVAL, dict(activation=3)), (EINVAL, dict(activation=-1)),
    (EINVAL, dict(workspace=P + 8)), (EUNSUPPORTED, dict(dtype=0)), (EUNSUPPORTED, dict(K=60)), (EUNSUPPORTED, dict(N=70)),
    (EOVERFLOW, dict(C=1 << 31)), (EOVERFLOW, dict(C=1 << 30, N=1 << 20)),
]


@pytest.mark.parametrize("rc,change", LINEAR_BAD + [
    (EINVAL, dict(y=None)), (EINVAL, dict(y=P + 8)), (EINVAL, dict(bias=P + 4)), (EINVAL, dict(residual=P + 2)), (EINVAL, dict(y=Q[5])),
    (EINVAL, dict(y=Q[0])), (EINVAL, dict(z=Q[0])), (ESMALLBUF, dict(C=100, K=8192, workspace=None)),
    (ESMALLBUF, dict(C=100, K=8192, workspace_bytes=64)),
])
def test_linear_fwd_refuses(rc, change):
    assert L.lib().harts_linear_fwd(ctypes.byref(_args(L.LinearArgs, LINEAR, **change)), None) == rc
    assert L.lib().harts_last_error()


@pytest.mark.parametrize("rc,change", [(rc, _fwd(c)) for rc, c in LINEAR_BAD] + [
    (EINVAL, dict(d_y=None)), (EINVAL, {"fwd.z": None}), (EINVAL, dict(d_y=P + 2)), (EINVAL, dict(dx=P + 8)), (EINVAL, dict(dweight=P + 8)),
    (EINVAL, dict(dbias=P + 4)), (EINVAL, dict(dx=None, dweight=None, dbias=None)), (EINVAL, dict(dx=Q[0])), (EINVAL, dict(dx=Q[6])),
    (EINVAL, dict(dweight=Q[1])), (EINVAL, dict(dweight=Q[5])), (EINVAL, dict(dweight=Q[7])), (ESMALLBUF, {"fwd.workspace": None}),
    (ESMALLBUF, {"fwd.workspace_bytes": 64}), (EINVAL, {"fwd.workspace": P + 16}),
])
def test_linear_bwd_refuses(rc, change):
    assert L.lib().harts_linear_bwd(ctypes.byref(_args(L.LinearBwdArgs, LINEAR_BWD, **change)), None) == rc


def test_null_args_and_sizes():
    lib = L.lib()
    for f in (lib.harts_block_norm_fwd, lib.harts_block_norm_bwd, lib.harts_linear_fwd, lib.harts_linear_bwd):
        assert f(None, None) == EINVAL
    nb = lib.harts_block_norm_bwd_workspace_bytes
    assert nb(-1, 64, 1) == nb(4, 8193, 1) == nb(4, 0, 1) == nb(4, 64, 2) == 0 and nb(0, 64, 1) > 0
    f, b = lib.harts_linear_fwd_workspace_bytes, lib.harts_linear_bwd_workspace_bytes
    assert f(-1, 64, 64) == f(4, 60, 64) == f(4, 64, 0) == 0 and f(100, 8192, 72) > 0
    assert b(-1, 64, 64, 0, 1) == b(4, 64, 64, 3, 1) == 0 and b(300, 64, 72, 2, 1) >= 2 * 300 * 72 + 4 * 72
    # an empty call of a forward is complete without a pointer
    assert lib.harts_block_norm_fwd(ctypes.byref(_args(L.BlockNormArgs, dict(C=0, D=64, dtype=1, scale=1.0))), None) == 0
    assert lib.harts_linear_fwd(ctypes.byref(_args(L.LinearArgs, dict(C=0, K=64, N=64, dtype=1))), None) == 0


def test_python_checks():
    from prefix_shared_chunkwise_gb300 import api
    bf = torch.bfloat16
    x, w = torch.zeros(18, 64, dtype=bf), torch.zeros(64)
    pl = api.Plan([-1, 0, 0], [5, 6, 7], 64)
    with pytest.raises(ValueError, match="form"):
        api.scan_fwd(pl, x, x, form="sum")
    with pytest.raises(ValueError, match="rows"):
        api.scan_fwd(pl, x[:3], x[:3])
    with pytest.raises(ValueError, match="g has"):
        api.scan_fwd(pl, x, x.float())
    with pytest.raises(ValueError, match="contiguous"):
        api.scan_fwd(pl, torch.zeros(64, 18, dtype=bf).t(), x)
    with pytest.raises(ValueError, match="h0"):
        api.scan_fwd(pl, x, x, h0=torch.zeros(2, 64))
    with pytest.raises(ValueError, match="final_state"):
        api.scan_fwd(pl, x, x, final_state=torch.zeros(2, 64, dtype=bf))
    with pytest.raises(ValueError, match="d_h"):
        api.scan_bwd(pl, x, x, x, x[:4])
    with pytest.raises(ValueError, match="d_final"):
        api.scan_bwd(pl, x, x, x, x, d_final=torch.zeros(3, 64))
    with pytest.raises(ValueError, match="unsupported dtype"):
        api.scan_fwd(pl, x.half(), x.half())
    with pytest.raises(ValueError, match="gate_act"):
        api.block_norm_fwd(x, post_weight=w, gate=x, gate_act="relu")
    with pytest.raises(ValueError, match="residual"):
        api.block_norm_fwd(x, post_weight=w, residual=x[:2])
    with pytest.raises(ValueError, match="pre_weight"):
        api.block_norm_fwd(x, pre_weight=w.bfloat16())
    with pytest.raises(ValueError, match="go with pre_weight"):
        api.block_norm_fwd(x, post_weight=w, n=x)
    with pytest.raises(ValueError, match="d_n"):
        api.block_norm_bwd(x, x, x[:2], post_weight=w, pre_weight=w)
    with pytest.raises(ValueError, match="activation"):
        api.linear_fwd(x, x, activation="relu")
    with pytest.raises(ValueError, match="weight"):
        api.linear_fwd(x, x[:, :32])
    with pytest.raises(ValueError, match="bias"):
        api.linear_fwd(x, x, torch.zeros(18, dtype=bf))
    with pytest.raises(ValueError, match="d_y"):
        api.linear_bwd(x, x, x)
    with pytest.raises(ValueError, match="expected a CUDA device"):
        api.linear_fwd(x, torch.zeros(24, 64, dtype=bf))


def _tiles(parent, seg_len, rows=128):
    """The scan's tiles by their definition: (segment, tile) in the order of segments."""
    return [(v, t) for v, n in enumerate(seg_len) for t in range((n + rows - 1) // rows)]


def test_workspace_holds_every_tile_and_group():
    """fp32 states of every group of 8 tiles (longer groups are fewer) and pairs of every tile of 128 rows, 64 bf16 or 32 fp32 channels wide."""
    from prefix_shared_chunkwise_gb300.api import Plan
    r = np.random.default_rng(3)
    for _ in range(20):
        n = int(r.integers(2, 30))
        parent = [-1] + [int(r.integers(0, i)) for i in range(1, n)]
        length = [int(v) for v in r.integers(1, 9000, n)]
        pl = Plan(parent, length, 64)
        tiles = len(_tiles(parent, length))
        groups = sum((v + 1023) // 1024 for v in length)
        up = lambda b: (b + 255) // 256 * 256
        for D, dtype, width in ((64, 1, 64), (72, 1, 128), (72, 0, 96), (1000, 0, 1024)):
            assert L.lib().harts_scan_workspace_bytes(pl.handle, D, dtype) == 256 + up(4 * width * groups) + up(8 * width * tiles)
