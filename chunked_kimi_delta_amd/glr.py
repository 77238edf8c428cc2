"""The gated linear recurrence with one state a channel (include/glr.h): argument marshalling only, as
in api.py."""
from __future__ import annotations

import ctypes

import torch

from ._lib import GlrArgs, load
from .api import _GATES, _INT32, _IO, _call, _check, _on, _ptr


def _rows(t, name, dtype, shape, device):
    """Checks a tensor [B, T, D] whose tokens may be columns of wider rows, of a longer batch; elements from token to
    token, and from row to row of the batch (0: T tokens)."""
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name}: expected device {device}, got {t.device}")
    if t.is_contiguous():
        return shape[2], 0
    B, T, D = shape
    per = t.stride(1) if T > 1 else D
    batch = t.stride(0) if B > 1 else 0
    if (D > 1 and t.stride(2) != 1) or per < D or (B > 1 and batch < (T - 1) * per + D):
        raise ValueError(f"{name}: channels must be contiguous, tokens evenly spaced and rows of the batch one behind another")
    return per, batch


def _arguments(x, g, beta, cu_seqlens, initial_state, use_beta_sigmoid, gate, A_log, dt_bias, gate_lower_bound):
    """Checked glr_args of the inputs (x may be None); y and the final state are the caller's to set."""
    dt, dev = g.dtype, g.device
    if dt not in _IO:
        raise TypeError(f"unsupported io dtype {dt} (bf16 or fp32)")
    if g.dim() != 3:
        raise ValueError("x, g and beta must be [B, T, D]")
    B, T, D = shape = g.shape
    if B > _INT32 or T > _INT32 or D > _INT32:
        raise ValueError(f"B, T and D are at most 2^31 - 1 (got {B}, {T}, {D})")
    if dev.type != "cuda":
        raise ValueError("inputs must be on a HIP device")
    gs, gb = _rows(g, "g", dt, shape, dev)
    xs, xb = (D, 0) if x is None else _rows(x, "x", dt, shape, dev)
    bs, bb = (D, 0) if beta is None else _rows(beta, "beta", dt, shape, dev)
    if use_beta_sigmoid and beta is None:
        raise ValueError("use_beta_sigmoid needs beta")
    N, cu, h0 = B, None, None
    if cu_seqlens is not None:
        if cu_seqlens.dtype != torch.int64 or cu_seqlens.device != dev or cu_seqlens.dim() != 1:
            raise ValueError("cu_seqlens must be a 1-D int64 tensor on the inputs' device")
        if not cu_seqlens.is_contiguous():
            raise ValueError("cu_seqlens must be contiguous")
        N, cu = cu_seqlens.numel() - 1, cu_seqlens.data_ptr()
        if N > _INT32:
            raise ValueError(f"at most 2^31 - 1 sequences (got {N})")
    if initial_state is not None:
        _check(initial_state, "initial_state", torch.float32, (N, D), dev)
        h0 = initial_state.data_ptr()
    if gate not in _GATES:
        raise ValueError(f"gate must be None, 'softplus' or 'bounded' (got {gate!r})")
    A = bias = None
    if gate is not None:
        if A_log is None:
            raise ValueError("a gate needs A_log")
        _check(A_log, "A_log", torch.float32, (D,), dev)
        A = A_log.data_ptr()
        if dt_bias is not None:
            _check(dt_bias, "dt_bias", torch.float32, (D,), dev)
            bias = dt_bias.data_ptr()
    a = GlrArgs(B, T, N, D, _IO[dt], None if x is None else x.data_ptr(), g.data_ptr(),
                None if beta is None else beta.data_ptr(), xs, gs, bs, cu, h0, None, None,
                int(bool(use_beta_sigmoid)), _GATES[gate], float(gate_lower_bound), A, bias)
    if xb or gb or bb:
        a.x_batch, a.g_batch, a.beta_batch = xb, gb, bb
    return a


def _like(g):
    return torch.empty_like(g, memory_format=torch.contiguous_format)


def _workspace(given, need, dev):
    if given is None:
        return torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    _check(given, "workspace", torch.uint8, given.shape, dev)
    if given.numel() < need:
        raise ValueError(f"workspace too small: {given.numel()} < {need} bytes")
    return given


class GlrFwdPlan:
    """Validated arguments for repeated glr_fwd calls on the same tensors:
    h <- exp(g) h + beta x, y = h, with one state a channel.

    x, g, beta [B,T,D] (all bf16 or all fp32, on one HIP device; beta None: ones): g is the log decay.
    They may be columns of wider rows (slices of one projection) and some tokens of a longer batch. cu_seqlens int64 [N+1] on the device
    (then B == 1) or None; initial_state fp32 [N,D] or None. Outputs y (contiguous, like x) and
    final_state (fp32 [N,D], or None; may be initial_state) are allocated once and reused by every
    call(). Any D up to 2^18 and any length, zero included, in fewer than 2^23 pieces: sequences times
    ceil(D / 64) channels, or for long sequences 64 tokens of 64 channels (2^35 values). What infinities and log
    decays above zero give, and how far fp32 outputs err, is in include/glr.h.

    Pre-stage, done inside the kernels: use_beta_sigmoid takes beta as logits; gate "softplus"
    (g <- -exp(A_log) softplus(g + dt_bias)) or "bounded" (g <- gate_lower_bound * sigmoid(exp(A_log)
    (g + dt_bias))) takes g as the raw gate input, with A_log fp32 [D] and dt_bias fp32 [D] or None.
    """

    def __init__(self, x, g, beta=None, cu_seqlens=None, initial_state=None, output_final_state=True,
                 workspace=None, y=None, final_state=None, use_beta_sigmoid=False, gate=None, A_log=None,
                 dt_bias=None, gate_lower_bound=-5.0):
        self.lib = load()
        a = _arguments(x, g, beta, cu_seqlens, initial_state, use_beta_sigmoid, gate, A_log, dt_bias,
                       gate_lower_bound)
        dev = self.device = g.device
        self.y = _like(g) if y is None else y
        if y is not None:
            _check(y, "y", g.dtype, g.shape, dev)
        a.y = self.y.data_ptr()
        self.final_state = None
        if output_final_state:
            self.final_state = (torch.empty((a.N, a.D), dtype=torch.float32, device=dev)
                                if final_state is None else final_state)
            if final_state is not None:
                _check(final_state, "final_state", torch.float32, (a.N, a.D), dev)
            a.final_state = self.final_state.data_ptr()
        self.args = a
        self.workspace = _workspace(workspace, _on(dev, self.lib.glr_fwd_workspace_bytes, ctypes.byref(a)), dev)
        self._ptrs = (ctypes.byref(a), *((None, 0) if self.workspace is None else
                                         (self.workspace.data_ptr(), self.workspace.numel())))
        self._keep = (x, g, beta, cu_seqlens, initial_state, A_log, dt_bias)

    def __call__(self, stream=None):
        """Enqueue the forward on `stream` (default: torch's current stream)."""
        _call(self.lib.glr_fwd, "glr_fwd", self.device, stream, *self._ptrs)
        return self.y, self.final_state


def glr_fwd(x, g, beta=None, cu_seqlens=None, initial_state=None, output_final_state=True, workspace=None,
            **prestage):
    """Gated linear recurrence forward. Returns (y, final_state or None; rows of y behind the last packed
    sequence hold anything); see GlrFwdPlan for shapes and the pre-stage keywords (use_beta_sigmoid, gate,
    A_log, dt_bias, gate_lower_bound)."""
    return GlrFwdPlan(x, g, beta, cu_seqlens, initial_state, output_final_state, workspace, **prestage)()


class GlrBwdPlan:
    """Validated arguments for repeated glr_bwd calls: gradients of glr_fwd with respect to x, g, beta,
    initial_state and (with a gate) A_log, dt_bias, from d_y (like y) and dht (fp32 [N,D] or None).

    y is the forward's output as it returned it (the states that g's gradient takes); x is read with beta
    only and may be None without. Other inputs as for GlrFwdPlan. Outputs, allocated once and reused by
    every call(): dx, dg, dbeta (with beta) in the io dtype, contiguous; dh0 fp32 [N,D] (when want_dh0),
    dA_log and ddt_bias fp32 [D] (with a gate).
    """

    def __init__(self, x, g, y, d_y, beta=None, dht=None, cu_seqlens=None, initial_state=None, want_dh0=True,
                 workspace=None, use_beta_sigmoid=False, gate=None, A_log=None, dt_bias=None,
                 gate_lower_bound=-5.0):
        self.lib = load()
        if x is None and beta is not None:
            raise ValueError("with beta, x is needed")
        a = _arguments(x, g, beta, cu_seqlens, initial_state, use_beta_sigmoid, gate, A_log, dt_bias,
                       gate_lower_bound)
        dev = self.device = g.device
        _check(y, "y", g.dtype, g.shape, dev)
        _check(d_y, "d_y", g.dtype, g.shape, dev)
        if dht is not None:
            _check(dht, "dht", torch.float32, (a.N, a.D), dev)
        a.y = y.data_ptr()
        f32 = dict(dtype=torch.float32, device=dev)
        self.dx, self.dg, self.dbeta = _like(g), _like(g), None if beta is None else _like(g)
        self.dh0 = torch.empty((a.N, a.D), **f32) if want_dh0 else None
        self.dA_log = torch.empty(a.D, **f32) if gate is not None else None
        self.ddt_bias = torch.empty(a.D, **f32) if gate is not None else None
        self.args = a
        self.workspace = _workspace(workspace, _on(dev, self.lib.glr_bwd_workspace_bytes, ctypes.byref(a)), dev)
        self._outs = (self.dx, self.dg, self.dbeta, self.dh0, self.dA_log, self.ddt_bias)
        self._ptrs = (ctypes.byref(a), _ptr(d_y), _ptr(dht),
                      *((None, 0) if self.workspace is None else (self.workspace.data_ptr(), self.workspace.numel())),
                      *map(_ptr, self._outs))
        self._keep = (x, g, y, d_y, beta, dht, cu_seqlens, initial_state, A_log, dt_bias)

    def __call__(self, stream=None):
        """Enqueue the backward on `stream` (default: torch's current stream); returns
        (dx, dg, dbeta, dh0, dA_log, ddt_bias)."""
        _call(self.lib.glr_bwd, "glr_bwd", self.device, stream, *self._ptrs)
        return self._outs


def glr_bwd(x, g, y, d_y, beta=None, dht=None, cu_seqlens=None, initial_state=None, want_dh0=True, **prestage):
    """Gated linear recurrence backward. Returns (dx, dg, dbeta or None in the io dtype, dh0 fp32 or None,
    dA_log or None, ddt_bias or None; rows behind the last packed sequence hold anything); see GlrBwdPlan. y and d_y
    are copied where they are not contiguous."""
    return GlrBwdPlan(x, g, y.contiguous(), d_y.contiguous(), beta, dht, cu_seqlens, initial_state, want_dh0, **prestage)()


class GlrStepPlan:
    """Validated arguments for repeated glr_step calls on the same tensors (a serving loop that writes
    each step's inputs in place).

    x, g, beta [B,T,D]: T new tokens of B rows (beta None: ones); state fp32 [slots,D], updated in place;
    state_indices int32 [B] on the device, or None for slot b of row b. A row whose index is negative or
    >= slots is padding: zeros in y, no state touched. Indices of other rows must differ. y [B,T,D] is
    allocated once and reused. Pre-stage keywords as for GlrFwdPlan.
    """

    def __init__(self, x, g, state, beta=None, state_indices=None, y=None, use_beta_sigmoid=False, gate=None,
                 A_log=None, dt_bias=None, gate_lower_bound=-5.0):
        self.lib = load()
        if state.shape[0] > _INT32:
            raise ValueError(f"at most 2^31 - 1 slots (got {state.shape[0]})")
        a = _arguments(x, g, beta, None, None, use_beta_sigmoid, gate, A_log, dt_bias, gate_lower_bound)
        self.device = g.device
        _check(state, "state", torch.float32, (state.shape[0], a.D), g.device)
        if state_indices is not None:
            _check(state_indices, "state_indices", torch.int32, (a.B,), g.device)
        elif state.shape[0] < a.B:
            raise ValueError(f"state has {state.shape[0]} slots for {a.B} rows")
        self.y = _like(g) if y is None else y
        if y is not None:
            _check(y, "y", g.dtype, g.shape, g.device)
        a.y = self.y.data_ptr()
        self.args = a
        self._call = (ctypes.byref(a), state.data_ptr(), _ptr(state_indices), state.shape[0])
        self._keep = (x, g, beta, state, state_indices, A_log, dt_bias)

    def __call__(self, stream=None):
        """Enqueue the step on `stream` (default: torch's current stream)."""
        _call(self.lib.glr_step, "glr_step", self.device, stream, *self._call)
        return self.y


def glr_step(x, g, state, beta=None, state_indices=None, **prestage):
    """A serving step of the gated linear recurrence: returns y and updates `state` in place; see
    GlrStepPlan."""
    return GlrStepPlan(x, g, state, beta, state_indices, **prestage)()
