"""What the update-tail entry points refuse, on the host: every case returns its error code
before anything is enqueued, so none of them needs a GPU."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from prefix_shared_chunkwise_gb300 import _lib as L

P = 1 << 20          # a well-aligned address that is never dereferenced
EINVAL, EUNSUPPORTED, EOVERFLOW, ESMALLBUF = -1, -2, -3, -4


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


NORM = dict(C=4, D=64, dtype=1, eps=1e-6, x=P, weight=P, y=P)
NORM_BWD = dict(C=4, D=64, dtype=1, dy=P, h=P, weight=P, rstd=P, dx=P, dweight=P, workspace=P,
                workspace_bytes=1 << 30)
HEAD = dict(C=4, V=100, D=64, dtype=1, scale=1.0, S=5, x=P, weight=P, row_ptr=P, row_sem=P, target=P, lse=P,
            logp=P, workspace=P, workspace_bytes=1 << 30)


@pytest.mark.parametrize("rc,change", [
    (EINVAL, dict(x=None)), (EINVAL, dict(weight=None)), (EINVAL, dict(y=None)), (EINVAL, dict(x=P + 8)),
    (EINVAL, dict(y=P + 2)), (EINVAL, dict(residual=P)), (EINVAL, dict(residual=P + 4, h=P)), (EINVAL, dict(C=-1)),
    (EINVAL, dict(D=0)), (EINVAL, dict(eps=-1.0)), (EINVAL, dict(eps=float("nan"))), (EINVAL, dict(eps=float("inf"))),
    (EINVAL, dict(y8=P)), (EINVAL, dict(y8_scale=P)), (EUNSUPPORTED, dict(dtype=2)), (EUNSUPPORTED, dict(dtype=-1)),
    (EUNSUPPORTED, dict(D=16385)), (EUNSUPPORTED, dict(D=48, y8=P, y8_scale=P)),
])
def test_rmsnorm_fwd_refuses(rc, change):
    assert L.lib().harts_rmsnorm_fwd(ctypes.byref(_args(L.RmsnormFwdArgs, NORM, **change)), None) == rc
    assert L.lib().harts_last_error()


@pytest.mark.parametrize("rc,change", [
    (EINVAL, dict(dy=None)), (EINVAL, dict(h=None)), (EINVAL, dict(weight=None)), (EINVAL, dict(rstd=None)),
    (EINVAL, dict(dx=None)), (EINVAL, dict(dweight=None)), (EINVAL, dict(dh=P + 2)), (EINVAL, dict(dx=P + 8)),
    (ESMALLBUF, dict(workspace=None)), (ESMALLBUF, dict(workspace_bytes=8)), (EUNSUPPORTED, dict(dtype=7)),
    (EUNSUPPORTED, dict(D=20000)), (EINVAL, dict(C=-2)),
])
def test_rmsnorm_bwd_refuses(rc, change):
    assert L.lib().harts_rmsnorm_bwd(ctypes.byref(_args(L.RmsnormBwdArgs, NORM_BWD, **change)), None) == rc


def test_null_args_and_sizes():
    lib = L.lib()
    assert lib.harts_rmsnorm_fwd(None, None) == EINVAL and lib.harts_rmsnorm_bwd(None, None) == EINVAL
    assert lib.harts_linear_logprob_fwd(None, None) == EINVAL and lib.harts_linear_logprob_bwd(None, None) == EINVAL
    assert lib.harts_rmsnorm_bwd_workspace_bytes(-1, 64, 1) == 0
    assert lib.harts_rmsnorm_bwd_workspace_bytes(4, 16385, 1) == 0
    assert lib.harts_linear_logprob_fwd_workspace_bytes(4, 0, 64) == 0
    assert lib.harts_linear_logprob_bwd_workspace_bytes(4, 10, 64, 5, -1) == 0
    assert lib.harts_grad_workspace_bytes(-1) == 0 and lib.harts_grad_workspace_bytes(0) > 0
    # an empty call of either forward is complete without a pointer
    assert lib.harts_rmsnorm_fwd(ctypes.byref(_args(L.RmsnormFwdArgs, dict(C=0, D=64, dtype=1, eps=1e-6))), None) == 0
    empty = _args(L.LinearLogprobFwdArgs, dict(C=0, V=10, D=64, dtype=1, scale=1.0, S=0))
    assert lib.harts_linear_logprob_fwd(ctypes.byref(empty), None) == 0


@pytest.mark.parametrize("rc,change", [
    (EINVAL, dict(x=None)), (EINVAL, dict(weight=None)), (EINVAL, dict(row_ptr=None)), (EINVAL, dict(row_sem=None)),
    (EINVAL, dict(target=None)), (EINVAL, dict(lse=None)), (EINVAL, dict(logp=None)), (EINVAL, dict(x=P + 8)),
    (EINVAL, dict(weight=P + 4)), (EINVAL, dict(V=0)), (EINVAL, dict(C=-1)), (EINVAL, dict(S=-1)),
    (EINVAL, dict(scale=float("inf"))), (EINVAL, dict(scale=float("nan"))), (EUNSUPPORTED, dict(dtype=0)),
    (EUNSUPPORTED, dict(D=60)), (EOVERFLOW, dict(S=1 << 31)), (EOVERFLOW, dict(C=1 << 31)),
    (ESMALLBUF, dict(workspace=None)), (ESMALLBUF, dict(workspace_bytes=16)),
])
def test_linear_logprob_fwd_refuses(rc, change):
    assert L.lib().harts_linear_logprob_fwd(ctypes.byref(_args(L.LinearLogprobFwdArgs, HEAD, **change)), None) == rc


@pytest.mark.parametrize("rc,change", [
    (EINVAL, dict(dlogp=None)), (EINVAL, dict(dx=None)), (EINVAL, dict(dweight=None)), (EINVAL, dict(piece=-1)),
    (EINVAL, dict(dx=P + 2)), (EINVAL, dict(dweight=P + 8)), (EINVAL, {"fwd.lse": None}),
    (EUNSUPPORTED, {"fwd.dtype": 0}), (ESMALLBUF, {"fwd.workspace_bytes": 16}), (EINVAL, {"fwd.workspace": P + 16}),
])
def test_linear_logprob_bwd_refuses(rc, change):
    base = {**{f"fwd.{k}": v for k, v in HEAD.items()}, "dlogp": P, "dx": P, "dweight": P, "piece": 0}
    assert L.lib().harts_linear_logprob_bwd(ctypes.byref(_args(L.LinearLogprobBwdArgs, base, **change)), None) == rc


GRAD = dict(g=P, out=P, n=10, dtype=1, out_dtype=1)


@pytest.mark.parametrize("rc,change", [
    (EINVAL, dict(g=None)), (EINVAL, dict(out=None)), (EINVAL, dict(n=-1)), (EINVAL, dict(g=P + 1)),
    (EINVAL, dict(out=P + 1)), (EINVAL, dict(dtype=0, g=P + 2)), (EINVAL, dict(out_dtype=0)),
    (EUNSUPPORTED, dict(dtype=3)), (EUNSUPPORTED, dict(out_dtype=3)), (EOVERFLOW, dict(n=(1 << 44) + 1)),
])
def test_grad_clip_refuses(rc, change):
    t = (L.GradTensor * 1)(_args(L.GradTensor, GRAD, **change))
    assert L.lib().harts_grad_clip(t, 1, 1.0, P, P, 1 << 20, None) == rc


def test_grad_call_refuses():
    lib, t = L.lib(), (L.GradTensor * 1)(_args(L.GradTensor, GRAD))
    assert lib.harts_grad_clip(t, -1, 1.0, P, P, 1 << 20, None) == EINVAL
    assert lib.harts_grad_clip(None, 1, 1.0, P, P, 1 << 20, None) == EINVAL
    assert lib.harts_grad_clip(t, 1, -1.0, P, P, 1 << 20, None) == EINVAL
    assert lib.harts_grad_clip(t, 1, float("nan"), P, P, 1 << 20, None) == EINVAL
    assert lib.harts_grad_clip(t, 1, 1.0, None, P, 1 << 20, None) == EINVAL
    assert lib.harts_grad_clip(t, 1, 1.0, P, P, 8, None) == ESMALLBUF
    assert lib.harts_grad_clip(t, 1, 1.0, P, P + 4, 1 << 20, None) == EINVAL
    assert lib.harts_grad_norm(t, 1, P, None, 0, None) == ESMALLBUF


def test_python_checks():
    from prefix_shared_chunkwise_gb300 import api
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(64)
    with pytest.raises(ValueError, match="contiguous"):
        api.rmsnorm_fwd(torch.zeros(64, 4, dtype=torch.bfloat16).t(), w)
    with pytest.raises(ValueError, match="weight"):
        api.rmsnorm_fwd(x, w.bfloat16())
    with pytest.raises(ValueError, match="residual"):
        api.rmsnorm_fwd(x, w, x[:2])
    with pytest.raises(ValueError, match="multiple of 32"):
        api.rmsnorm_fwd(x[:, :40].contiguous(), w[:40], mx8=True)
    with pytest.raises(ValueError, match="dtype"):
        api.rmsnorm_fwd(x.half(), w)
    with pytest.raises(ValueError, match="rstd"):
        api.rmsnorm_bwd(x, x, w, torch.zeros(3))
    i = torch.zeros(5, dtype=torch.int32)
    head = torch.zeros(100, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="weight"):
        api.linear_logprob_fwd(x, head[:, :32], i, i, i)
    with pytest.raises(ValueError, match="row_sem"):
        api.linear_logprob_fwd(x, head, i, i.long(), i)
    with pytest.raises(ValueError, match="dlogp"):
        api.linear_logprob_bwd(x, head, i, i, i, torch.zeros(4), torch.zeros(4))
    with pytest.raises(ValueError, match="outputs"):
        api.GradSet([x], [])
    with pytest.raises(ValueError, match="output 0"):
        api.GradSet([x], [x[:2]])
    with pytest.raises(ValueError, match="unsupported dtype"):
        api.GradSet([x.half()])


def test_linear_logprob_positions_up_to_the_last_step_of_an_index():
    """The kernels step up to 256 past the last position in 32 bits: 2^31 - 256 is the most.  A
    count that is taken gets as far as the workspace's size."""
    def call(S):
        a = _args(L.LinearLogprobFwdArgs, HEAD, S=S, workspace_bytes=16)
        return L.lib().harts_linear_logprob_fwd(ctypes.byref(a), None)
    assert call((1 << 31) - 256) == ESMALLBUF
    assert call((1 << 31) - 255) == EOVERFLOW and call((1 << 31) - 1) == EOVERFLOW


def test_grad_workspace_of_the_most_tensors():
    """A partial sum for each block of each launch of 512 tensors, whatever the count."""
    nb = L.lib().harts_grad_workspace_bytes
    per = nb(512)
    assert per > 256 and nb(513) == 2 * per
    for count in ((1 << 31) - 1, (1 << 31) - 511, 1 << 30):
        assert nb(count) == (count + 511) // 512 * per


class _Tensor:
    """What the choice of a stream asks of a tensor, without a GPU."""
    is_cuda, device = True, "cuda:1"

    def get_device(self):
        return 1


class _Stream:
    cuda_stream = 77

    def __init__(self, device_index):
        self.device_index = device_index


def test_other_devices_are_refused(monkeypatch):
    """Kernels start on the current device: with tensors or a stream of another one they would run
    there, on the wrong GPU's addresses."""
    from prefix_shared_chunkwise_gb300 import api
    t, now = _Tensor(), [1]
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 100 + dev, raising=False)
    for stream_of in (api._stream_on, lambda s, t: api._stream(s, t).value):
        now[0] = 1
        assert stream_of(None, t) == 101 and stream_of(_Stream(1), t) == 77
        with pytest.raises(ValueError, match="stream is on cuda:0"):
            stream_of(_Stream(0), t)
        now[0] = 0
        with pytest.raises(ValueError, match="current device is cuda:0"):
            stream_of(None, t)
        with pytest.raises(ValueError, match="current device is cuda:0"):
            stream_of(_Stream(1), t)
    with pytest.raises(ValueError, match="expected a CUDA device"):
        api._stream_on(None, torch.zeros(1))


def test_rmsnorm_fwd_refuses_one_buffer_for_both_outputs():
    for residual in (None, P):
        a = _args(L.RmsnormFwdArgs, NORM, x=2 * P, residual=residual, h=P, y=P)
        assert L.lib().harts_rmsnorm_fwd(ctypes.byref(a), None) == EINVAL
