"""Thin Python binding over the C ABI: the same calls, with torch tensors for device
memory and streams.  Every step of the computation runs in the library's kernels;
this module only marshals pointers and sizes."""
from __future__ import annotations

import ctypes
import functools

import numpy as np

from . import _lib as L

__all__ = ["Plan", "kda_fwd", "kda_bwd", "conv_fwd", "conv_bwd", "semantic_map", "logprob_fwd",
           "logprob_bwd", "attn_fwd", "attn_bwd", "linear_logprob_fwd", "linear_logprob_bwd",
           "rmsnorm_fwd", "rmsnorm_bwd", "GradSet", "device_error", "dtype_code"]


def dtype_code(torch_dtype):
    import torch
    if torch_dtype == torch.float32:
        return L.HARTS_FP32
    if torch_dtype == torch.bfloat16:
        return L.HARTS_BF16
    raise ValueError(f"unsupported dtype {torch_dtype}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream, t=None):
    """The raw handle of the given stream, or of the current one.  `t`: a tensor of the call,
    see _stream_on."""
    import torch
    if t is not None and t.is_cuda:
        return ctypes.c_void_p(_stream_on(stream, t))
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _made_on_stream(call):
    """Runs `call` under the stream it is given, if any, so that the buffers it makes belong to
    that stream: a workspace made on the current one would be handed out again, as soon as the
    call returns, to work that does not wait for this stream's kernels."""
    @functools.wraps(call)
    def run(*args, stream=None, **kw):
        if stream is None:
            return call(*args, **kw)
        import torch
        with torch.cuda.stream(stream):
            return call(*args, stream=stream, **kw)
    return run


class Plan:
    """harts_plan_calls + harts_plan_get_info / export / upload / free.

    nodewise=True asks for the node-wise plan (HARTS_PLAN_NODEWISE): one sequence per
    segment, one round per tree level.  noreplay=True asks for the no-replay plan
    (HARTS_PLAN_NOREPLAY, forward only): side branches start from the exact fork state."""

    def __init__(self, parent, seg_len, chunk: int, nodewise: bool = False, noreplay: bool = False):
        parent = np.ascontiguousarray(parent, np.int32)
        seg_len = np.ascontiguousarray(seg_len, np.int64)
        h = ctypes.c_void_p()
        flags = (L.HARTS_PLAN_NODEWISE if nodewise else 0) | (L.HARTS_PLAN_NOREPLAY if noreplay else 0)
        rc = L.lib().harts_plan_calls(len(parent), parent.ctypes.data_as(L._pi32),
                                      seg_len.ctypes.data_as(L._pi64), int(chunk), flags,
                                      ctypes.byref(h))
        L.check(rc, "harts_plan_calls")
        self._h = h
        info = L.PlanInfo()
        L.check(L.lib().harts_plan_get_info(self._h, ctypes.byref(info)), "harts_plan_get_info")
        self.info = {n: getattr(info, n) for n, _ in L.PlanInfo._fields_}
        self._dev = None

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value:
            L.lib().harts_plan_free(h)
            self._h = None

    @property
    def handle(self):
        return self._h

    def arrays(self) -> dict:
        """Export every plan array into numpy (harts_plan_export)."""
        info = self.info
        env = dict(info)
        out, arr = {}, L.PlanArrays()
        for name, ty, size in L.PLAN_ARRAY_FIELDS:
            n = eval(size, {}, env)
            a = np.zeros(max(n, 1), np.int64 if ty == "i64" else np.int32)
            out[name] = (a, n)
            setattr(arr, name, a.ctypes.data_as(L._pi64 if ty == "i64" else L._pi32))
        L.check(L.lib().harts_plan_export(self._h, ctypes.byref(arr)), "harts_plan_export")
        return {k: a[:n] for k, (a, n) in out.items()}

    def device_bytes(self) -> int:
        return int(L.lib().harts_plan_device_bytes(self._h))

    def upload(self, device="cuda", stream=None):
        """Allocate the plan's device tables through torch and upload them."""
        import torch
        nb = self.device_bytes()
        with torch.cuda.stream(stream):             # None: the current one
            buf = torch.empty(nb, dtype=torch.uint8, device=device)
        L.check(L.lib().harts_plan_upload(self._h, _ptr(buf), nb, _stream(stream, buf)),
                "harts_plan_upload")
        self._dev = buf
        return self

    def device_error(self, stream=None) -> int:
        code = ctypes.c_int32(0)
        rc = L.lib().harts_plan_device_error(self._h, _stream(stream, self._dev), ctypes.byref(code))
        if rc not in (0, -7):
            L.check(rc, "harts_plan_device_error")
        return code.value

    def chunk_state_bytes(self, H, dk, dv, dtype_c):
        return int(L.lib().harts_kda_chunk_state_bytes(self._h, H, dk, dv, dtype_c))

    def bwd_workspace_bytes(self, H, dk, dv):
        return int(L.lib().harts_kda_bwd_workspace_bytes(self._h, H, dk, dv))


def device_error(stream=None) -> int:
    """harts_device_error: waits for the stream; the code that a call without a plan and without
    an error word of its own left on the current device (3: a bounded wait ran out, its outputs are
    incomplete), or 0.  Reading clears it."""
    code = ctypes.c_int32(0)
    rc = L.lib().harts_device_error(_stream(stream), ctypes.byref(code))
    if rc not in (0, -7):
        L.check(rc, "harts_device_error")
    return code.value


def _need(name, t, shape=None, dtype=None, nbytes=None, device=None):
    """Size check of one buffer before its pointer crosses the C ABI (which cannot see sizes)."""
    if t is None:
        return
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if nbytes is not None and t.numel() * t.element_size() < nbytes:
        raise ValueError(f"{name} holds {t.numel() * t.element_size()} bytes, needs {nbytes}")


def _fwd_args(plan, q, k, v, g, beta, o, states, final_state, h0, chunk_states, scale, kernel):
    import torch
    C, H, dk = q.shape
    dv = v.shape[2]
    info, dev, f32 = plan.info, q.device, torch.float32
    if C != info["C"]:
        raise ValueError(f"q has {C} rows, the plan {info['C']}")
    for n, t, sh in (("k", k, (C, H, dk)), ("v", v, (C, H, dv)), ("g", g, (C, H, dk)),
                     ("beta", beta, (C, H)), ("o", o, (C, H, dv))):
        _need(n, t, sh, q.dtype, device=dev)
    per = H * dk * dv * 4                          # bytes of one fp32 state, all heads
    _need("states", states, None, f32, info["n_states"] * per, dev)
    _need("final_state", final_state, None, f32, info["n_seq"] * per, dev)
    _need("h0", h0, None, f32, info["n_roots"] * per, dev)
    _need("chunk_states", chunk_states, nbytes=plan.chunk_state_bytes(H, dk, dv, dtype_code(q.dtype)),
          device=dev)
    a = L.FwdArgs()
    a.H, a.dk, a.dv = H, dk, dv
    a.dtype = dtype_code(q.dtype)
    a.kernel = kernel
    a.scale = float(scale)
    for n, t in dict(q=q, k=k, v=v, g=g, beta=beta, o=o, states=states, final_state=final_state,
                     h0=h0, chunk_states=chunk_states).items():
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
        setattr(a, n, None if t is None else t.data_ptr())
    return a


@_made_on_stream
def kda_fwd(plan: Plan, q, k, v, g, beta, *, o=None, states=None, final_state=None, h0=None,
            chunk_states=None, scale=1.0, kernel=L.HARTS_KERNEL_AUTO, stream=None):
    """harts_kda_fwd.  Allocates any missing output through torch; returns
    (o, states, final_state, chunk_states)."""
    import torch
    C, H, dk = q.shape
    dv = v.shape[2]
    info = plan.info
    dev = q.device
    if o is None:
        o = torch.empty((C, H, dv), dtype=q.dtype, device=dev)
    if states is None and info["n_states"] > 0:
        states = torch.empty((info["n_states"], H, dk, dv), dtype=torch.float32, device=dev)
    a = _fwd_args(plan, q, k, v, g, beta, o, states, final_state, h0, chunk_states, scale, kernel)
    L.check(L.lib().harts_kda_fwd(plan.handle, ctypes.byref(a), _stream(stream, q)), "harts_kda_fwd")
    return o, states, final_state, chunk_states


@_made_on_stream
def kda_bwd(plan: Plan, q, k, v, g, beta, d_o, *, states, chunk_states, d_final=None,
            h0=None, dh0=None, scale=1.0, grads=None, workspace=None,
            kernel=L.HARTS_KERNEL_AUTO, stream=None, phase="all"):
    """harts_kda_bwd (phase "all"), harts_kda_bwd_state ("state"), harts_kda_bwd_grad
    ("grad"), or harts_kda_bwd_static ("static": no workspace, the library's own scratch).
    Returns dict(dq, dk, dv, dg, dbeta[, dh0])."""
    import torch
    C, H, dk = q.shape
    dv = v.shape[2]
    dev = q.device
    if grads is None:
        grads = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
                     dg=torch.empty_like(g), dbeta=torch.empty_like(beta))
    nb = plan.bwd_workspace_bytes(H, dk, dv)
    if workspace is None and phase != "static":
        workspace = torch.empty(max(nb, 256), dtype=torch.uint8, device=dev)
    info = plan.info
    _need("d_o", d_o, (C, H, dv), q.dtype, device=dev)
    per = H * dk * dv * 4
    _need("d_final", d_final, None, torch.float32, info["n_seq"] * per, dev)
    _need("dh0", dh0, None, torch.float32, info["n_roots"] * per, dev)
    for n, ref in (("dq", q), ("dk", k), ("dv", v), ("dg", g), ("dbeta", beta)):
        _need(n, grads[n], tuple(ref.shape), q.dtype, device=dev)
    if phase != "static":
        _need("workspace", workspace, nbytes=nb, device=dev)
    a = L.BwdArgs()
    a.fwd = _fwd_args(plan, q, k, v, g, beta, None, states, None, h0, chunk_states, scale, kernel)
    a.d_o = d_o.data_ptr()
    a.d_final = None if d_final is None else d_final.data_ptr()
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        setattr(a, n, grads[n].data_ptr())
    a.dh0 = None if dh0 is None else dh0.data_ptr()
    a.workspace = None if workspace is None else workspace.data_ptr()
    a.workspace_bytes = 0 if workspace is None else workspace.numel()
    fn = {"all": "harts_kda_bwd", "state": "harts_kda_bwd_state", "grad": "harts_kda_bwd_grad",
          "static": "harts_kda_bwd_static"}[phase]
    L.check(getattr(L.lib(), fn)(plan.handle, ctypes.byref(a), _stream(stream, q)), fn)
    if dh0 is not None:
        grads["dh0"] = dh0
    return grads


def _conv_args(x, weight, bias, y, activation):
    C, ch = x.shape[0], int(x.numel() // x.shape[0])
    a = L.ConvFwdArgs()
    a.channels, a.width = ch, int(weight.shape[1])
    a.dtype = dtype_code(x.dtype)
    a.activation = {"none": 0, "silu": 1}[activation]
    for n, t in dict(x=x, weight=weight, bias=bias, y=y).items():
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
        setattr(a, n, None if t is None else t.data_ptr())
    return a


@_made_on_stream
def conv_fwd(plan: Plan, x, weight, bias=None, *, activation="none", y=None, stream=None):
    """harts_conv_fwd.  x: [C, ...] compact rows (channels = the rest, flattened);
    weight: [channels, w] fp32; bias: [channels] fp32 or None.  Returns y like x."""
    import torch
    if y is None:
        y = torch.empty_like(x)
    a = _conv_args(x, weight, bias, y, activation)
    L.check(L.lib().harts_conv_fwd(plan.handle, ctypes.byref(a), _stream(stream, x)), "harts_conv_fwd")
    return y


@_made_on_stream
def conv_bwd(plan: Plan, x, weight, bias, dy, *, activation="none", dx=None, dweight=None, dbias=None,
             workspace=None, stream=None):
    """harts_conv_bwd.  Returns (dx, dweight, dbias); dbias is None when bias is None."""
    import torch
    if dx is None:
        dx = torch.empty_like(x)
    if dweight is None:
        dweight = torch.empty_like(weight)
    if dbias is None and bias is not None:
        dbias = torch.empty_like(bias)
    b = L.ConvBwdArgs()
    b.fwd = _conv_args(x, weight, bias, None, activation)
    nb = int(L.lib().harts_conv_bwd_workspace_bytes(plan.handle, b.fwd.channels, b.fwd.width))
    if workspace is None:
        workspace = torch.empty(max(nb, 256), dtype=torch.uint8, device=x.device)
    b.dy, b.dx, b.dweight = dy.data_ptr(), dx.data_ptr(), dweight.data_ptr()
    b.dbias = None if dbias is None else dbias.data_ptr()
    b.workspace, b.workspace_bytes = workspace.data_ptr(), workspace.numel()
    L.check(L.lib().harts_conv_bwd(plan.handle, ctypes.byref(b), _stream(stream, x)), "harts_conv_bwd")
    return dx, dweight, dbias


def semantic_map(plan: Plan):
    """harts_plan_semantic_map: numpy (sem_row [S], row_ptr [C+1], row_sem [S]) int32."""
    C, S = plan.info["C"], plan.info["S"]
    sem_row = np.zeros(max(S, 1), np.int32)
    row_ptr = np.zeros(C + 1, np.int32)
    row_sem = np.zeros(max(S, 1), np.int32)
    L.check(L.lib().harts_plan_semantic_map(plan.handle, sem_row.ctypes.data_as(L._pi32),
                                            row_ptr.ctypes.data_as(L._pi32), row_sem.ctypes.data_as(L._pi32)),
            "harts_plan_semantic_map")
    return sem_row[:S], row_ptr, row_sem[:S]


def _lp_args(logits, row_ptr, row_sem, target, lse, logp):
    a = L.LogprobFwdArgs()
    a.C, a.V = logits.shape
    a.dtype = dtype_code(logits.dtype)
    a.S = target.numel()
    for n, t in dict(logits=logits, row_ptr=row_ptr, row_sem=row_sem, target=target, lse=lse, logp=logp).items():
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
        setattr(a, n, None if t is None else t.data_ptr())
    return a


@_made_on_stream
def logprob_fwd(logits, row_ptr, row_sem, target, *, lse=None, logp=None, stream=None):
    """harts_logprob_fwd: returns (logp [S] fp32, lse [C] fp32)."""
    import torch
    if lse is None:
        lse = torch.empty(logits.shape[0], dtype=torch.float32, device=logits.device)
    if logp is None:
        logp = torch.empty(target.numel(), dtype=torch.float32, device=logits.device)
    a = _lp_args(logits, row_ptr, row_sem, target, lse, logp)
    L.check(L.lib().harts_logprob_fwd(ctypes.byref(a), _stream(stream, logits)), "harts_logprob_fwd")
    return logp, lse


@_made_on_stream
def logprob_bwd(logits, row_ptr, row_sem, target, lse, dlogp, *, dlogits=None, stream=None):
    """harts_logprob_bwd: returns dlogits like logits."""
    import torch
    if dlogits is None:
        dlogits = torch.empty_like(logits)
    b = L.LogprobBwdArgs()
    b.fwd = _lp_args(logits, row_ptr, row_sem, target, lse, None)
    b.dlogp, b.dlogits = dlogp.data_ptr(), dlogits.data_ptr()
    L.check(L.lib().harts_logprob_bwd(ctypes.byref(b), _stream(stream, logits)), "harts_logprob_bwd")
    return dlogits


@_made_on_stream
def attn_fwd(plan: Plan, q, k, v, *, scale=None, o=None, lse=None, stream=None):
    """harts_attn_fwd: branch attention over the compact layout.  q, k, v: [C, H, d]
    bf16 (d = 128).  Returns (o [C, H, d] bf16, lse [C, H] fp32)."""
    import torch
    C, H, d = q.shape
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((C, H), dtype=torch.float32, device=q.device)
    for n, t in dict(q=q, k=k, v=v, o=o, lse=lse).items():
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    a = _attn_args(q, k, v, o, lse, scale)
    L.check(L.lib().harts_attn_fwd(plan.handle, ctypes.byref(a), _stream(stream, q)), "harts_attn_fwd")
    return o, lse


def _attn_args(q, k, v, o, lse, scale):
    C, H, d = q.shape
    a = L.AttnFwdArgs()
    a.H, a.d, a.dtype = H, d, dtype_code(q.dtype)
    a.scale = float(d ** -0.5 if scale is None else scale)
    a.q, a.k, a.v, a.o = q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr()
    a.lse = None if lse is None else lse.data_ptr()
    return a


@_made_on_stream
def attn_bwd(plan: Plan, q, k, v, o, lse, d_o, *, scale=None, dq=None, dk=None, dv=None, workspace=None,
             stream=None):
    """harts_attn_bwd: returns (dq, dk, dv) like q, from the forward's o and lse."""
    import torch
    for n, t in dict(q=q, k=k, v=v, o=o, lse=lse, d_o=d_o).items():
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    b = L.AttnBwdArgs()
    b.fwd = _attn_args(q, k, v, o, lse, scale)
    nb = int(L.lib().harts_attn_bwd_workspace_bytes(plan.handle, q.shape[1]))
    if workspace is None:
        workspace = torch.empty(max(nb, 256), dtype=torch.uint8, device=q.device)
    b.d_o, b.dq, b.dk, b.dv = d_o.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr()
    b.workspace, b.workspace_bytes = workspace.data_ptr(), workspace.numel()
    L.check(L.lib().harts_attn_bwd(plan.handle, ctypes.byref(b), _stream(stream, q)), "harts_attn_bwd")
    return dq, dk, dv


def _stream_on(stream, t):
    """The raw handle of the given stream, or of the current one of `t`'s device (without
    building a Stream object: this runs in every call, some of which take a few us).  The library
    launches on the current device: tensors and streams of another one are refused."""
    if not t.is_cuda:
        raise ValueError(f"tensors are on {t.device}, expected a CUDA device")
    import torch
    dev, now = t.get_device(), torch.cuda.current_device()
    if stream is not None and stream.device_index != dev:
        raise ValueError(f"stream is on cuda:{stream.device_index}, tensors are on cuda:{dev}")
    if dev != now:
        raise ValueError(f"tensors are on cuda:{dev}, the current device is cuda:{now} (torch.cuda.device)")
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _ready(name, t, shape, dtype, device):
    """_need, and contiguous: what every buffer that a caller gives to the operators below has
    to be.  None is an absent buffer; a shape of None is not compared."""
    if t is None or (t.dtype is dtype and t.device == device and t.is_contiguous()
                     and (shape is None or t.shape == shape)):
        return
    _need(name, t, shape, dtype, None, device)
    raise ValueError(f"{name} must be contiguous")


@_made_on_stream
def rmsnorm_fwd(x, weight, residual=None, *, eps=1e-6, mx8=False, y=None, h=None, rstd=None, stream=None):
    """harts_rmsnorm_fwd: h = x + residual, y = h / sqrt(mean h^2 + eps) * weight per row.
    x, residual: [C, D] bf16 or fp32; weight: [D] fp32.  Returns (y, h, rstd [C] fp32).  mx8=True
    returns y as (values [C, D] float8_e4m3fn, scales [C, D/32] float8_e8m0fnu) instead; D is
    then a multiple of 32.  h may be given as x or residual, y as x (in place).  Without a
    residual a given h receives x; with none given, h is x itself, or None where y is written
    over it (nothing is left for the backward)."""
    import torch
    shape, dt, dev, f32 = x.shape, x.dtype, x.device, torch.float32
    if len(shape) != 2:
        raise ValueError(f"x has shape {tuple(shape)}, expected [C, D]")
    C, D = shape
    code = dtype_code(dt)
    _ready("x", x, None, dt, dev)
    _ready("weight", weight, (D,), f32, dev)
    y_ptr = q_ptr = scale_ptr = res_ptr = h_ptr = None
    if mx8:
        if D % 32:
            raise ValueError("mx8 needs D a multiple of 32")
        if y is None:
            y = (torch.empty(shape, dtype=torch.float8_e4m3fn, device=dev),
                 torch.empty((C, D // 32), dtype=torch.float8_e8m0fnu, device=dev))
        else:
            _ready("y values", y[0], shape, torch.float8_e4m3fn, dev)
            _ready("y scales", y[1], (C, D // 32), torch.float8_e8m0fnu, dev)
        q_ptr, scale_ptr = y[0].data_ptr(), y[1].data_ptr()
    else:
        if y is None:
            y = torch.empty_like(x)
        else:
            _ready("y", y, shape, dt, dev)
        y_ptr = y.data_ptr()
    if h is not None:
        _ready("h", h, shape, dt, dev)
        h_ptr = h.data_ptr()
    if residual is not None:
        _ready("residual", residual, shape, dt, dev)
        if h is None:
            h = torch.empty_like(x)
            h_ptr = h.data_ptr()
        res_ptr = residual.data_ptr()
    elif h is None and (C == 0 or y_ptr != x.data_ptr()):
        h = x
    if rstd is None:
        rstd = torch.empty(C, dtype=f32, device=dev)
    else:
        _ready("rstd", rstd, (C,), f32, dev)
    a = L.RmsnormFwdArgs(C, D, code, eps, x.data_ptr(), res_ptr, weight.data_ptr(), h_ptr, y_ptr, q_ptr, scale_ptr,
                         rstd.data_ptr())
    L.check(L.lib().harts_rmsnorm_fwd(ctypes.byref(a), _stream_on(stream, x)), "harts_rmsnorm_fwd")
    return y, h, rstd


@_made_on_stream
def rmsnorm_bwd(dy, h, weight, rstd, dh=None, *, dx=None, dweight=None, error=None, workspace=None, stream=None):
    """harts_rmsnorm_bwd: from dL/dy, the forward's h and rstd, and dL/dh along the residual
    stream (or None).  Returns (dx [C, D] like h: the gradient of x and of the residual;
    dweight [D] fp32).  error: as linear_logprob_fwd's."""
    import torch
    shape, dt, dev, f32 = h.shape, h.dtype, h.device, torch.float32
    if len(shape) != 2:
        raise ValueError(f"h has shape {tuple(shape)}, expected [C, D]")
    C, D = shape
    code = dtype_code(dt)
    _ready("h", h, None, dt, dev)
    _ready("dy", dy, shape, dt, dev)
    _ready("dh", dh, shape, dt, dev)
    _ready("weight", weight, (D,), f32, dev)
    _ready("rstd", rstd, (C,), f32, dev)
    if dx is None:
        dx = torch.empty_like(h)
    else:
        _ready("dx", dx, shape, dt, dev)
    if dweight is None:
        dweight = torch.empty(D, dtype=f32, device=dev)
    else:
        _ready("dweight", dweight, (D,), f32, dev)
    _need("error", error, None, torch.int32, 4, dev)
    lib = L.lib()
    nb = lib.harts_rmsnorm_bwd_workspace_bytes(C, D, code)
    workspace, nb = _workspace(workspace, nb, dev)
    a = L.RmsnormBwdArgs(C, D, code, dy.data_ptr(), h.data_ptr(), None if dh is None else dh.data_ptr(),
                         weight.data_ptr(), rstd.data_ptr(), dx.data_ptr(), dweight.data_ptr(),
                         None if error is None else error.data_ptr(), workspace.data_ptr(), nb)
    L.check(lib.harts_rmsnorm_bwd(ctypes.byref(a), _stream_on(stream, h)), "harts_rmsnorm_bwd")
    return dx, dweight


def _workspace(workspace, nb, dev):
    """The caller's workspace, or one of `nb` bytes; and its size."""
    if workspace is None:
        import torch
        return torch.empty(max(nb, 256), dtype=torch.uint8, device=dev), max(nb, 256)
    _need("workspace", workspace, nbytes=nb, device=dev)
    return workspace, workspace.numel() * workspace.element_size()


class GradSet:
    """harts_grad_norm / harts_grad_clip over a fixed list of gradient buffers (bf16 or fp32,
    contiguous, one device).  The buffers and their addresses are taken once and kept; their values
    are read at every call.  A program whose gradients are new tensors each step (autograd's after
    grad = None) needs a new set each step: an old one goes on clipping the buffers it was made of.
    outs: where clip() writes (same shapes, bf16 or fp32), None: in place.
    A set outlives the graphs that its calls were captured into, and its calls run one after
    another: they share its workspace."""

    def __init__(self, grads, outs=None):
        import torch
        grads = list(grads)
        outs = grads if outs is None else list(outs)
        if len(outs) != len(grads):
            raise ValueError(f"{len(outs)} outputs for {len(grads)} gradients")
        self.grads, self.outs = grads, outs
        self._dev = grads[0].device if grads else torch.empty(0, device="cuda").device
        self._list = (L.GradTensor * max(len(grads), 1))()
        for i, (g, o) in enumerate(zip(grads, outs)):
            _ready(f"gradient {i}", g, None, g.dtype, self._dev)
            _ready(f"output {i}", o, g.shape, o.dtype, self._dev)
            t = self._list[i]
            t.g, t.out, t.n = g.data_ptr(), o.data_ptr(), g.numel()
            t.dtype, t.out_dtype = dtype_code(g.dtype), dtype_code(o.dtype)
        self._ws, self._nb = _workspace(None, L.lib().harts_grad_workspace_bytes(len(grads)), self._dev)
        self._made_on = _stream_on(None, self._ws)

    def _call_stream(self, stream):
        """The call's raw stream; the workspace is not handed out again before it is done there."""
        raw = _stream_on(stream, self._ws)
        if raw != self._made_on:
            import torch
            self._ws.record_stream(torch.cuda.current_stream(self._dev))
        return raw

    def _norm(self, norm):
        import torch
        if norm is None:
            return torch.empty((), dtype=torch.float32, device=self._dev)
        _need("norm", norm, None, torch.float32, 4, self._dev)
        return norm

    @_made_on_stream
    def norm(self, *, norm=None, stream=None):
        """The global 2-norm, a 0-dim fp32 tensor."""
        norm = self._norm(norm)
        L.check(L.lib().harts_grad_norm(self._list, len(self.grads), norm.data_ptr(), self._ws.data_ptr(), self._nb,
                                        self._call_stream(stream)), "harts_grad_norm")
        return norm

    @_made_on_stream
    def clip(self, max_norm, *, norm=None, stream=None):
        """outs = grads * min(1, max_norm / norm); returns the norm before clipping."""
        norm = self._norm(norm)
        L.check(L.lib().harts_grad_clip(self._list, len(self.grads), max_norm, norm.data_ptr(), self._ws.data_ptr(),
                                        self._nb, self._call_stream(stream)), "harts_grad_clip")
        return norm


def _head_checks(x, weight, row_ptr, row_sem, target, error):
    """(C, V, D, S) of the operands that forward and backward share."""
    import torch
    if x.dim() != 2 or weight.dim() != 2:
        raise ValueError("x and weight must be [C, D] and [V, D]")
    (C, D), V, S, dt, dev, i32 = x.shape, weight.shape[0], target.numel(), x.dtype, x.device, torch.int32
    _ready("x", x, None, dt, dev)
    _ready("weight", weight, (V, D), dt, dev)
    _ready("row_ptr", row_ptr, (C + 1,), i32, dev)
    _ready("row_sem", row_sem, (S,), i32, dev)
    _ready("target", target, (S,), i32, dev)
    _need("error", error, None, i32, 4, dev)
    return C, V, D, S


@_made_on_stream
def linear_logprob_fwd(x, weight, row_ptr, row_sem, target, *, scale=1.0, lse=None, logp=None, error=None,
                       workspace=None, stream=None):
    """harts_linear_logprob_fwd: log-probabilities of the semantic positions from hidden rows
    x [C, D] and the vocabulary weight [V, D] (bf16), without forming the logits in memory.
    A target outside 0 .. V-1 has no label (logp 0).  Returns (logp [S] fp32, lse [C] fp32).
    error: int32 device tensor that a bounded wait which ran out sets to 3; None: the library's own
    word, see device_error()."""
    import torch
    C, V, D, S = _head_checks(x, weight, row_ptr, row_sem, target, error)
    dev, f32 = x.device, torch.float32
    if lse is None:
        lse = torch.empty(C, dtype=f32, device=dev)
    else:
        _ready("lse", lse, (C,), f32, dev)
    if logp is None:
        logp = torch.empty(S, dtype=f32, device=dev)
    else:
        _ready("logp", logp, (S,), f32, dev)
    lib = L.lib()
    workspace, nb = _workspace(workspace, lib.harts_linear_logprob_fwd_workspace_bytes(C, V, D), dev)
    a = L.LinearLogprobFwdArgs(C, V, D, dtype_code(x.dtype), scale, S, x.data_ptr(), weight.data_ptr(),
                               row_ptr.data_ptr(), row_sem.data_ptr(), target.data_ptr(), lse.data_ptr(),
                               logp.data_ptr(), None if error is None else error.data_ptr(), workspace.data_ptr(), nb)
    L.check(lib.harts_linear_logprob_fwd(ctypes.byref(a), _stream_on(stream, x)), "harts_linear_logprob_fwd")
    return logp, lse


@_made_on_stream
def linear_logprob_bwd(x, weight, row_ptr, row_sem, target, lse, dlogp, *, scale=1.0, dx=None, dweight=None,
                       piece=0, error=None, workspace=None, stream=None):
    """harts_linear_logprob_bwd: returns (dx like x, dweight like weight) from the forward's lse
    and dL/dlogp [S] fp32.  piece: vocabulary entries whose logit gradients are held at a time
    (0: the library's choice)."""
    import torch
    C, V, D, S = _head_checks(x, weight, row_ptr, row_sem, target, error)
    dt, dev, f32 = x.dtype, x.device, torch.float32
    _ready("lse", lse, (C,), f32, dev)
    _ready("dlogp", dlogp, (S,), f32, dev)
    if dx is None:
        dx = torch.empty_like(x)
    else:
        _ready("dx", dx, x.shape, dt, dev)
    if dweight is None:
        dweight = torch.empty_like(weight)
    else:
        _ready("dweight", dweight, weight.shape, dt, dev)
    lib = L.lib()
    workspace, nb = _workspace(workspace, lib.harts_linear_logprob_bwd_workspace_bytes(C, V, D, S, max(piece, 0)), dev)
    f = L.LinearLogprobFwdArgs(C, V, D, dtype_code(dt), scale, S, x.data_ptr(), weight.data_ptr(), row_ptr.data_ptr(),
                               row_sem.data_ptr(), target.data_ptr(), lse.data_ptr(), None,
                               None if error is None else error.data_ptr(), workspace.data_ptr(), nb)
    a = L.LinearLogprobBwdArgs(f, dlogp.data_ptr(), dx.data_ptr(), dweight.data_ptr(), piece)
    L.check(lib.harts_linear_logprob_bwd(ctypes.byref(a), _stream_on(stream, x)), "harts_linear_logprob_bwd")
    return dx, dweight
