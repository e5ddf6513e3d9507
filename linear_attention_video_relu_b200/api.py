"""Torch-facing wrapper of the C ABI: tensors in, tensors out.

PyTorch provides device memory and streams only; the computation is the
CUDA library's. Shapes follow include/linattn.h: q, k, v, gate, out are
contiguous [B, H, N, D] (layout="bhnd") or [B, N, H, D] (layout="bnhd") in
bf16 or fp32; the carried state is fp32 S [B, H, D, D] and z [B, H, D].
"""
from __future__ import annotations

import contextlib
from typing import Optional, Sequence

import torch

from . import _native as C

_DTYPES = {torch.bfloat16: C.LA_BF16, torch.float32: C.LA_F32}
_MODES = {"bidirectional": C.LA_BIDIRECTIONAL, "block_causal": C.LA_BLOCK_CAUSAL,
          "token_causal": C.LA_TOKEN_CAUSAL}
_LAYOUTS = {"bhnd": C.LA_LAYOUT_BHND, "bnhd": C.LA_LAYOUT_BNHD}


def _dims(t: torch.Tensor, layout: str):
    """(B, H, N, D) of a [B, H, N, D] or [B, N, H, D] tensor."""
    if layout not in _LAYOUTS:
        raise ValueError("layout must be 'bhnd' or 'bnhd'")
    if t.dim() != 4:
        raise ValueError("expected a 4D tensor, got shape %s" % (tuple(t.shape),))
    a, b, c, d = t.shape
    return (a, b, c, d) if layout == "bhnd" else (a, c, b, d)


def make_params(B: int, H: int, N: int, D: int, dtype: torch.dtype, mode: str = "bidirectional",
                block_tokens: int = 0, grid: Optional[Sequence[int]] = None,
                rope_split: Optional[Sequence[int]] = None, theta: float = 10000.0,
                eps: float = 1e-6, layout: str = "bhnd") -> C.la_params:
    p = C.la_params()
    p.B, p.H, p.N, p.D = B, H, N, D
    if dtype not in _DTYPES:
        raise TypeError("dtype must be torch.bfloat16 or torch.float32")
    p.dtype = _DTYPES[dtype]
    p.mode = _MODES[mode]
    p.block_tokens = block_tokens
    p.rope = 1 if grid is not None else 0
    if grid is not None:
        p.grid_t, p.grid_h, p.grid_w = (int(x) for x in grid)
        p.rope_dt, p.rope_dh, p.rope_dw = (int(x) for x in rope_split)
    p.rope_theta = float(theta)
    p.eps = float(eps)
    if layout not in _LAYOUTS:
        raise ValueError("layout must be 'bhnd' or 'bnhd'")
    p.layout = _LAYOUTS[layout]
    return p


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


# torch's raw current-stream query, when this torch has it: the handle without
# building a Stream object (a per-call cost on the host)
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
# the current device's index without the checks of torch.cuda.current_device
# (a CUDA tensor is at hand wherever this is asked, so CUDA is initialised)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _stream(stream: Optional[torch.cuda.Stream], device: Optional[int] = None):
    """The handle of `stream`, else of the current stream of `device` (an
    index; None: the current device)."""
    if stream is not None:
        return stream.cuda_stream
    if device is None:
        device = torch.cuda.current_device()
    if _current_raw_stream is not None:
        return _current_raw_stream(device)
    return torch.cuda.current_stream(device).cuda_stream


_same = contextlib.nullcontext()


def _on_device(t: torch.Tensor):
    """t's device made current for the call; no switch when it already is, nor for
    host tensors (which the checks of the call refuse)."""
    idx = t.get_device()
    if idx < 0 or idx == _current_device():
        return _same
    return torch.cuda.device(idx)


def _on_stream(t: torch.Tensor, stream: Optional[torch.cuda.Stream], makes: bool = True):
    """_on_device(t) for a call that also makes its results or its workspace:
    with a stream given, that is current for the call, so that they are filled
    on it and the allocator hands their memory on in its order. A call that
    `makes` nothing need not switch."""
    if stream is None:
        return _on_device(t)
    if stream.device != t.device:
        raise ValueError("the stream is on %s, the tensors on %s" % (stream.device, t.device))
    return torch.cuda.stream(stream) if makes else _on_device(t)


def _int32(x, what):
    """x, which the C side's int has to hold (ctypes would cut it off)."""
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError("%s must fit a 32-bit int, got %s" % (what, x))
    return x


_DTYPE_OF = {v: k for k, v in _DTYPES.items()}


def _same_device(ref: torch.Tensor, *ts):
    for t in ts:
        if t is not None and t.device != ref.device:
            raise ValueError("all tensors must be on %s, got one on %s" % (ref.device, t.device))


def _check_io(p: C.la_params, *ts, require_cuda: bool = True):
    """Contiguous CUDA tensors of shape [B, H, N, D] (or [B, N, H, D]) in the
    params' dtype (require_cuda=False checks the rest on host tensors)."""
    shape = ((p.B, p.H, p.N, p.D) if p.layout == C.LA_LAYOUT_BHND else (p.B, p.N, p.H, p.D))
    dt = _DTYPE_OF[p.dtype]
    for t in ts:
        if t is None:
            continue
        if t.dtype is dt and t.is_contiguous() and t.shape == shape and (t.is_cuda or
                                                                         not require_cuda):
            continue
        if (require_cuda and not t.is_cuda) or not t.is_contiguous():
            raise ValueError("tensors must be contiguous CUDA tensors")
        if tuple(t.shape) != shape:
            raise ValueError("expected shape %s, got %s" % (shape, tuple(t.shape)))
        if t.dtype != _DTYPE_OF[p.dtype]:
            raise TypeError("expected dtype %s, got %s" % (_DTYPE_OF[p.dtype], t.dtype))


class Workspace:
    """A device scratch buffer sized by the library, zeroed once: its leading
    control block must be zero before the first call, and every call leaves it
    zero."""

    def __init__(self, nbytes: int, device):
        self.nbytes = max(int(nbytes), 256)
        self.buf = torch.zeros(self.nbytes, dtype=torch.uint8, device=device)

    @property
    def ptr(self):
        return self.buf.data_ptr()

    def control_block_is_zero(self) -> bool:
        n = min(self.nbytes, C.LA_WORKSPACE_CONTROL_BYTES)
        return int(torch.count_nonzero(self.buf[:n])) == 0

    def status(self, stream=None) -> int:
        """Synchronise and read the bounded-wait flag (see lin_attn_device_status)."""
        return C.lin_attn_device_status(self.ptr, _stream(stream))


def workspace_for(p: C.la_params, device, block_step: bool = False) -> Workspace:
    with torch.cuda.device(device):
        n = C.lin_attn_block_step_workspace_size(p) if block_step else C.lin_attn_workspace_size(p)
    return Workspace(n, device)


def forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, gate: Optional[torch.Tensor] = None,
            *, mode: str = "bidirectional", block_tokens: int = 0,
            grid: Optional[Sequence[int]] = None, rope_split: Optional[Sequence[int]] = None,
            theta: float = 10000.0, eps: float = 1e-6, out: Optional[torch.Tensor] = None,
            workspace: Optional[Workspace] = None, stream=None,
            layout: str = "bhnd") -> torch.Tensor:
    """out = RoPE(phi q) S / (phi q . z + eps) [* sigmoid(gate)] over [B, H, N, D]
    tensors (or [B, N, H, D] ones with layout="bnhd")."""
    B, H, N, D = _dims(q, layout)
    p = make_params(B, H, N, D, q.dtype, mode, block_tokens, grid, rope_split, theta, eps,
                    layout)
    _check_io(p, q, k, v, gate)
    with _on_stream(q, stream, out is None or workspace is None):
        if out is None:
            out = torch.empty_like(q)
        _check_io(p, out)
        _same_device(q, k, v, gate, out, None if workspace is None else workspace.buf)
        if workspace is None:
            workspace = workspace_for(p, q.device)
        C.check(C.lin_attn_forward(p, _ptr(q), _ptr(k), _ptr(v), _ptr(gate), _ptr(out),
                                   workspace.ptr, workspace.nbytes,
                                   _stream(stream, q.get_device())), "lin_attn_forward")
    return out


def cross_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                  gate: Optional[torch.Tensor] = None, *, eps: float = 1e-6,
                  out: Optional[torch.Tensor] = None, workspace: Optional[Workspace] = None,
                  stream=None, layout: str = "bhnd") -> torch.Tensor:
    """Linear cross-attention: q, gate, out [B, H, N, D] read the state of
    k, v [B, H, M, D] (no RoPE; every query sees every key); [B, N, H, D] and
    [B, M, H, D] with layout="bnhd"."""
    B, H, N, D = _dims(q, layout)
    kB, kH, M, kD = _dims(k, layout)
    if (kB, kH, kD) != (B, H, D):
        raise ValueError("k must have q's B, H and D; got shape %s" % (tuple(k.shape),))
    p = make_params(B, H, N, D, q.dtype, eps=eps, layout=layout)
    pk = make_params(B, H, M, D, q.dtype, eps=eps, layout=layout)
    _check_io(p, q, gate)
    _check_io(pk, k, v)
    with _on_stream(q, stream, out is None or workspace is None):
        if out is None:
            out = torch.empty_like(q)
        _check_io(p, out)
        _same_device(q, k, v, gate, out, None if workspace is None else workspace.buf)
        if workspace is None:
            workspace = Workspace(C.lin_attn_cross_workspace_size(p, M), q.device)
        C.check(C.lin_attn_cross_forward(p, M, _ptr(q), _ptr(k), _ptr(v), _ptr(gate), _ptr(out),
                                         workspace.ptr, workspace.nbytes,
                                         _stream(stream, q.get_device())),
                "lin_attn_cross_forward")
    return out


class BlockState:
    """The constant-memory cache (S, z) of block-causal generation."""

    def __init__(self, B: int, H: int, D: int, device="cuda"):
        self.S = torch.zeros((B, H, D, D), dtype=torch.float32, device=device)
        self.z = torch.zeros((B, H, D), dtype=torch.float32, device=device)
        self.B, self.H, self.D = B, H, D
        self._st = C.la_state()
        C.check(C.lin_attn_state_init(self._st, B, H, D, self.S.data_ptr(), self.z.data_ptr()),
                "lin_attn_state_init")
        self._ws = {}
        self._plans = {}

    def reset(self, stream=None) -> None:
        with torch.cuda.device(self.S.device):
            C.check(C.lin_attn_state_reset(self._st, _stream(stream)), "lin_attn_state_reset")

    def _workspace(self, p):
        key = (p.N, p.D, p.dtype, p.rope, p.grid_t, p.grid_h, p.grid_w, p.rope_dt, p.rope_dh,
               p.rope_dw, p.layout)
        ws = self._ws.get(key)
        if ws is None:
            ws = workspace_for(p, self.S.device, block_step=True)
            self._ws[key] = ws
        return ws

    def _plan(self, x, grid, rope_split, theta, eps, layout):
        """(params, workspace) of a block of x's shape and dtype with these
        settings, made once per distinct call and kept (params are only read
        by the library)."""
        key = (x.shape, x.dtype, None if grid is None else tuple(grid),
               None if rope_split is None else tuple(rope_split), theta, eps, layout)
        ent = self._plans.get(key)
        if ent is None:
            B, H, N, D = _dims(x, layout)
            p = make_params(B, H, N, D, x.dtype, "bidirectional", 0, grid, rope_split, theta,
                            eps, layout)
            ent = (p, self._workspace(p))
            self._plans[key] = ent
        return ent

    def step(self, q, k, v, gate=None, *, t_offset: int = 0, commit: bool = True,
             grid=None, rope_split=None, theta: float = 10000.0, eps: float = 1e-6,
             out=None, stream=None, layout: str = "bhnd") -> torch.Tensor:
        """One block of block-causal attention against the carried state."""
        _int32(t_offset, "t_offset")
        with _on_stream(self.S, stream):
            p, ws = self._plan(q, grid, rope_split, theta, eps, layout)
            _check_io(p, q, k, v, gate)
            if out is None:
                out = torch.empty_like(q)
            else:
                _check_io(p, out)
            _same_device(self.S, q, k, v, gate, out)
            dev = q.get_device()
            C.check(C.lin_attn_block_step(p, self._st, t_offset, q.data_ptr(), k.data_ptr(),
                                          v.data_ptr(), _ptr(gate), out.data_ptr(),
                                          1 if commit else 0, ws.ptr, ws.nbytes,
                                          _stream(stream, dev)), "lin_attn_block_step")
        return out

    def update(self, k, v, *, t_offset: int = 0, grid=None, rope_split=None,
               theta: float = 10000.0, stream=None, layout: str = "bhnd") -> None:
        """Fold a block's k, v into the state without producing output."""
        _int32(t_offset, "t_offset")
        with _on_stream(self.S, stream):
            p, ws = self._plan(k, grid, rope_split, theta, 1e-6, layout)
            _check_io(p, k, v)
            _same_device(self.S, k, v)
            C.check(C.lin_attn_state_update(p, self._st, t_offset, k.data_ptr(), v.data_ptr(),
                                            ws.ptr, ws.nbytes, _stream(stream, k.get_device())),
                    "lin_attn_state_update")


def uses_tensor_cores(B, H, N, D, dtype, **kw) -> bool:
    return bool(C.lin_attn_uses_tensor_cores(make_params(B, H, N, D, dtype, **kw)))


def temporal_conv(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                  cache_in: Optional[torch.Tensor] = None, *,
                  cache_out: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """Mix-FFN temporal convolution with the last-frame cache:
    y[t] = x[t] + w0 * x[t-1] + w1 * x[t] + w2 * x[t+1] (+ bias), per channel,
    with a zero frame after the block and cache_in (or zero) before it.

    x, out: [B, T, S, C] or [B, T, Hg, Wg, C] (bf16 or fp32); weight fp32
    [3, C]; bias fp32 [C]; cache_in, cache_out: one frame, [B, S, C] or
    [B, Hg, Wg, C], in x's dtype. cache_out receives x's last frame (it may be
    cache_in itself)."""
    if x.dim() not in (4, 5):
        raise ValueError("x must be [B, T, S, C] or [B, T, Hg, Wg, C]")
    if x.dtype not in _DTYPES:
        raise TypeError("x must be bf16 or fp32")
    B, T, nc = int(x.shape[0]), int(x.shape[1]), int(x.shape[-1])
    S = 1
    for d in x.shape[2:-1]:
        S *= int(d)
    frame_shape = (B,) + tuple(x.shape[2:])
    with _on_stream(x, stream, out is None):
        if out is None:
            out = torch.empty_like(x)
        for t, shape, dt, what in ((x, tuple(x.shape), x.dtype, "x"),
                                   (out, tuple(x.shape), x.dtype, "out"),
                                   (weight, (3, nc), torch.float32, "weight"),
                                   (bias, (nc,), torch.float32, "bias"),
                                   (cache_in, frame_shape, x.dtype, "cache_in"),
                                   (cache_out, frame_shape, x.dtype, "cache_out")):
            if t is None:
                continue
            if not t.is_cuda or not t.is_contiguous():
                raise ValueError("%s must be a contiguous CUDA tensor" % what)
            if tuple(t.shape) != shape or t.dtype != dt:
                raise ValueError("%s must be %s %s, got %s %s" % (what, shape, dt, tuple(t.shape),
                                                                t.dtype))
        _same_device(x, out, weight, bias, cache_in, cache_out)
        C.check(C.lin_attn_temporal_conv(B, T, S, nc, _DTYPES[x.dtype], _ptr(x), _ptr(weight),
                                         _ptr(bias), _ptr(cache_in), _ptr(out), _ptr(cache_out),
                                         _stream(stream)),
                "lin_attn_temporal_conv")
    return out


# ---- the gated delta rule ------------------------------------------------------

def _delta_params(q, k, v, log_decay, beta, scale, layout) -> C.la_delta_params:
    """Params of a call with these tensors, which are checked: contiguous, on
    one CUDA device, in one dtype, of matching shapes."""
    B, Hk, N, D = _dims(q, layout)
    vB, H, vN, Dv = _dims(v, layout)
    dt, dev = q.dtype, q.get_device()
    gates = (B, H, N) if layout == "bhnd" else (B, N, H)
    # one cheap test of everything, then the errors that name what is wrong
    if not (dt in _DTYPES and dev >= 0 and vB == B and vN == N and k.shape == q.shape and
            log_decay.shape == gates and beta.shape == gates and k.dtype is dt and
            v.dtype is dt and log_decay.dtype is dt and beta.dtype is dt and
            k.get_device() == dev and v.get_device() == dev and
            log_decay.get_device() == dev and beta.get_device() == dev and
            q.is_contiguous() and k.is_contiguous() and v.is_contiguous() and
            log_decay.is_contiguous() and beta.is_contiguous()):
        if dt not in _DTYPES:
            raise TypeError("dtype must be torch.bfloat16 or torch.float32")
        if (vB, vN) != (B, N):
            raise ValueError("v must have q's B and N; got shape %s" % (tuple(v.shape),))
        for t, shape, what in ((q, q.shape, "q"), (k, q.shape, "k"), (v, v.shape, "v"),
                               (log_decay, gates, "log_decay"), (beta, gates, "beta")):
            _check_tensor(t, shape, dt, dev, what)
    return C.la_delta_params(B, H, N, Hk, D, Dv, _DTYPES[dt], _LAYOUTS[layout],
                             D ** -0.5 if scale is None else scale)


def _check_tensor(t, shape, dtype, device, what):
    """A contiguous tensor of this shape and dtype on CUDA device `device` (its
    index): one cheap test, then the error that names what is wrong."""
    if (t.shape == shape and t.dtype is dtype and t.get_device() == device and device >= 0 and
            t.is_contiguous()):
        return
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("%s must be a contiguous CUDA tensor" % what)
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (what, tuple(shape), tuple(t.shape)))
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (what, dtype, t.dtype))
    raise ValueError("all tensors must be on cuda:%d, got one on %s" % (device, t.device))


def _check_delta_extras(p, dev, state, lengths, *states):
    shape = (p.B, p.H, p.D, p.Dv)
    for t, what in ((state, "state"),) + states:
        if t is not None:
            _check_tensor(t, shape, torch.float32, dev, what)
    if lengths is not None:
        _check_tensor(lengths, (p.B,), torch.int32, dev, "lengths")


def _delta_workspace(workspace, need, q):
    """(buffer, its bytes) of a call: the caller's Workspace, or one of `need`
    bytes on q's device (no part of a delta-rule workspace has to be zero)."""
    if workspace is not None:
        _same_device(q, workspace.buf)
        return workspace.buf, workspace.nbytes
    if need == 0:
        return None, 0
    return torch.empty(need, dtype=torch.uint8, device=q.device), need


def delta_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
                  beta: torch.Tensor, *, state: Optional[torch.Tensor] = None,
                  lengths: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                  out: Optional[torch.Tensor] = None, state_out: Optional[torch.Tensor] = None,
                  workspace: Optional[Workspace] = None, stream=None, layout: str = "bhnd"):
    """The gated delta rule over N tokens, from `state` (None: zeros):
        S <- exp(log_decay_t) S;  S <- S + beta_t k_t (v_t - S^T k_t)^T;
        out_t = scale S^T q_t.
    Returns (out, state_out).

    q, k: [B, Hk, N, D]; v, out: [B, H, N, Dv]; log_decay, beta: [B, H, N]
    (layout="bnhd": [B, N, Hk, D], [B, N, H, Dv], [B, N, H]), bf16 or fp32;
    value head h reads query and key head h // (H // Hk). state, state_out:
    fp32 [B, H, D, Dv]; state_out may be `state`, which then is updated in
    place. lengths: int32 [B], the tokens each sequence has; rows of `out`
    behind them are left as they were, and zero in an `out` made here. scale:
    D ** -0.5 unless given. workspace: at least lin_attn_delta_workspace_size
    bytes, made here unless given. stream: the call's, for what it makes too.
    Keys are taken as they are: normalise them first. The results are in no
    autograd graph, whatever q, k and the others require: delta_backward gives
    the gradients, to a torch.autograd.Function or to whoever calls it."""
    p = _delta_params(q, k, v, log_decay, beta, scale, layout)
    dev = q.get_device()
    with _on_stream(q, stream):
        if out is None:
            out = torch.empty_like(v) if lengths is None else torch.zeros_like(v)
        else:
            _check_tensor(out, v.shape, v.dtype, dev, "out")
        if state_out is None:
            state_out = torch.empty((p.B, p.H, p.D, p.Dv), dtype=torch.float32, device=q.device)
        _check_delta_extras(p, dev, state, lengths, (state_out, "state_out"))
        ws, nbytes = None, 0
        if p.N > C.LA_DELTA_STEP_TOKENS or workspace is not None:
            ws, nbytes = _delta_workspace(workspace, C.lin_attn_delta_workspace_size(p), q)
        C.check(C.lin_attn_delta_forward(p, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                         log_decay.data_ptr(), beta.data_ptr(), _ptr(state),
                                         _ptr(lengths), out.data_ptr(), state_out.data_ptr(),
                                         _ptr(ws), nbytes, _stream(stream, dev)),
                "lin_attn_delta_forward")
    return out, state_out


def delta_backward(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                   log_decay: torch.Tensor, beta: torch.Tensor, *,
                   state: Optional[torch.Tensor] = None,
                   dstate_out: Optional[torch.Tensor] = None,
                   lengths: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                   out: Optional[Sequence[torch.Tensor]] = None,
                   dstate: Optional[torch.Tensor] = None,
                   workspace: Optional[Workspace] = None, stream=None, layout: str = "bhnd"):
    """Gradients of delta_forward: from those of its results (dout, and
    dstate_out or None for zeros) to (dq, dk, dv, dlog_decay, dbeta, dstate),
    shaped and typed as the inputs; dstate, that of the initial state, is None
    unless `state` or `dstate` is given. All is made again from the inputs.

    out: five tensors to take dq, dk, dv, dlog_decay and dbeta; with lengths,
    rows behind them are left as they were there, and zero in tensors made
    here. dstate may be dstate_out itself; whether it is wanted may change the last
    bit of the other gradients in bf16 (linattn.h). workspace: at least
    lin_attn_delta_backward_workspace_size bytes (0.6 GB for 2 x 16 heads of 4096
    tokens, 128 x 128), made here unless given."""
    p = _delta_params(q, k, v, log_decay, beta, scale, layout)
    dev = q.get_device()
    _check_tensor(dout, v.shape, v.dtype, dev, "dout")
    like = (q, k, v, log_decay, beta)
    with _on_stream(q, stream):
        if out is None:
            out = tuple(torch.empty_like(t) for t in like)
            if lengths is not None:
                torch._foreach_zero_(out)   # in one launch
        else:
            out = tuple(out)
            if len(out) != 5:
                raise ValueError("out must be five tensors: dq, dk, dv, dlog_decay, dbeta")
            for t, x, what in zip(out, like, ("dq", "dk", "dv", "dlog_decay", "dbeta")):
                _check_tensor(t, x.shape, x.dtype, dev, what)
        if dstate is None and state is not None:
            dstate = torch.empty_like(state)
        _check_delta_extras(p, dev, state, lengths, (dstate_out, "dstate_out"),
                            (dstate, "dstate"))
        ws, nbytes = _delta_workspace(workspace, C.lin_attn_delta_backward_workspace_size(p), q)
        C.check(C.lin_attn_delta_backward(p, dout.data_ptr(), q.data_ptr(), k.data_ptr(),
                                          v.data_ptr(), log_decay.data_ptr(), beta.data_ptr(),
                                          _ptr(state), _ptr(dstate_out), _ptr(lengths),
                                          *(t.data_ptr() for t in out), _ptr(dstate), _ptr(ws),
                                          nbytes, _stream(stream, dev)),
                "lin_attn_delta_backward")
    return out + (dstate,)


class DeltaState:
    """The carried state of gated-delta-rule layers: fp32 S [B, H, D, Dv]."""

    def __init__(self, B: int, H: int, D: int, Dv: Optional[int] = None, device="cuda"):
        self.S = torch.zeros((B, H, D, D if Dv is None else Dv), dtype=torch.float32,
                             device=device)

    def reset(self) -> None:
        self.S.zero_()

    def step(self, q, k, v, log_decay, beta, **kw) -> torch.Tensor:
        """Run the tokens given (one, or a whole prompt) against the state,
        which they update in place; arguments as for delta_forward."""
        return delta_forward(q, k, v, log_decay, beta, state=self.S, state_out=self.S, **kw)[0]


# ---- rotary positions ------------------------------------------------------------

_STYLES = {"interleaved": C.LA_ROTARY_INTERLEAVED, "half": C.LA_ROTARY_HALF}
_SCALINGS = {"none": C.LA_ROTARY_NO_SCALING, "linear": C.LA_ROTARY_LINEAR,
             "ntk": C.LA_ROTARY_NTK, "by_parts": C.LA_ROTARY_BY_PARTS}


def rotary(q: torch.Tensor, k: Optional[torch.Tensor] = None, *,
           positions: Optional[torch.Tensor] = None, offset: int = 0,
           grid: Optional[Sequence[int]] = None, rope_split: Optional[Sequence[int]] = None,
           dim: Optional[int] = None, style: str = "interleaved", theta: float = 10000.0,
           scaling: str = "none", factor: float = 1.0, original_length: float = 0.0,
           low: float = 1.0, high: float = 32.0, amplitude: float = 1.0,
           out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None, stream=None,
           layout: str = "bhnd"):
    """Rotary positions in the first `dim` (default all) columns of q's and k's
    heads; returns the rotated q, or (q, k) where k is given.

    q: [B, H, N, D], k: [B, Hk, N, D] (layout="bnhd": [B, N, H, D]), bf16 or
    fp32. positions: int32 [N] or [B, N]; without them token n is at offset + n,
    or, with grid=(T, Hg, Wg) and rope_split widths, at its frame (+ offset),
    row and column in three segments of the columns. style: "interleaved"
    (pairs 2m, 2m + 1) or "half" (m, m + dim / 2). scaling: "none", "linear",
    "ntk" or "by_parts" (with original_length, low, high turns), by `factor`.
    amplitude multiplies the rotated columns. out, k_out may be q and k. The
    results are in no autograd graph: rotary_backward gives the gradients."""
    return _rotary(q, k, positions, offset, grid, rope_split, dim, style, theta, scaling, factor,
                   original_length, low, high, amplitude, out, k_out, stream, layout, 0)


def rotary_backward(dq: torch.Tensor, dk: Optional[torch.Tensor] = None, *,
                    positions: Optional[torch.Tensor] = None, offset: int = 0,
                    grid: Optional[Sequence[int]] = None,
                    rope_split: Optional[Sequence[int]] = None, dim: Optional[int] = None,
                    style: str = "interleaved", theta: float = 10000.0, scaling: str = "none",
                    factor: float = 1.0, original_length: float = 0.0, low: float = 1.0,
                    high: float = 32.0, amplitude: float = 1.0,
                    out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
                    stream=None, layout: str = "bhnd"):
    """Gradients of rotary's inputs from those of its results: the transposed
    rotation, with the arguments of the forward call."""
    return _rotary(dq, dk, positions, offset, grid, rope_split, dim, style, theta, scaling, factor,
                   original_length, low, high, amplitude, out, k_out, stream, layout, 1)


def _rotary(q, k, positions, offset, grid, rope_split, dim, style, theta, scaling, factor,
            original_length, low, high, amplitude, out, k_out, stream, layout, transpose):
    B, H, N, D = _dims(q, layout)
    dt, dev = q.dtype, q.get_device()
    if dt not in _DTYPES:
        raise TypeError("dtype must be torch.bfloat16 or torch.float32")
    if style not in _STYLES:
        raise ValueError("style must be 'interleaved' or 'half'")
    if scaling not in _SCALINGS:
        raise ValueError("scaling must be 'none', 'linear', 'ntk' or 'by_parts'")
    if (grid is None) != (rope_split is None):
        raise ValueError("grid and rope_split go together")
    offset, dim_ = _int32(offset, "offset"), D if dim is None else _int32(dim, "dim")
    p = C.la_rotary_params(B, H, 0, N, D, dim_, _DTYPES[dt],
                           _LAYOUTS[layout], _STYLES[style], _SCALINGS[scaling], transpose, 0,
                           offset, 0, 0, 0, 0, 0, 0, theta, factor, original_length, low, high,
                           amplitude)
    if grid is not None:
        if positions is not None:
            raise ValueError("positions and grid exclude each other")
        p.grid_t, p.grid_h, p.grid_w = (_int32(int(x), "grid") for x in grid)
        p.rope_dt, p.rope_dh, p.rope_dw = (_int32(int(x), "rope_split") for x in rope_split)
        if dim is None:
            p.dim = p.rope_dt + p.rope_dh + p.rope_dw
    if not (dev >= 0 and q.is_contiguous()):
        _check_tensor(q, q.shape, dt, dev, "q")
    with _on_stream(q, stream):
        if out is None:
            out = torch.empty_like(q)
        else:
            _check_tensor(out, q.shape, dt, dev, "out")
        if k is not None:
            kB, p.Hk, kN, kD = _dims(k, layout)
            if kB != B or kN != N or kD != D:
                raise ValueError("k must have q's B, N and D; got shape %s" % (tuple(k.shape),))
            if not (k.dtype is dt and k.get_device() == dev and k.is_contiguous()):
                _check_tensor(k, k.shape, dt, dev, "k")
            if k_out is None:
                k_out = torch.empty_like(k)
            else:
                _check_tensor(k_out, k.shape, dt, dev, "k_out")
        elif k_out is not None:
            raise ValueError("k_out without k")
        if positions is not None:
            p.positions_per_batch = 1 if positions.dim() == 2 else 0
            _check_tensor(positions, (B, N) if p.positions_per_batch else (N,), torch.int32, dev,
                          "positions")
        C.check(C.lin_attn_rotary(p, q.data_ptr(), _ptr(k), _ptr(positions), out.data_ptr(),
                                  _ptr(k_out), _stream(stream, dev)), "lin_attn_rotary")
    return out if k is None else (out, k_out)
