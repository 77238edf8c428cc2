"""The gated delta rule with one decay per token and value head (include/gdn.h): argument
marshalling only, as in api.py."""
from __future__ import annotations

import ctypes

import torch

from ._lib import GdnArgs, load
from .act8 import Packed8, _check_packed, unpack8
from .api import _GATES, _IO, _call, _check, _on, _ptr


def _arguments(q, k, v, g, beta, scale, cu_seqlens, initial_state, use_qk_l2norm,
               use_beta_sigmoid, gate, A_log, dt_bias, gate_lower_bound, io=None):
    """Checked gdn_args of the inputs; o and the final state are the caller's to set. io: the io dtype
    where q, k and v are the int8 rows of checkpoints."""
    dt, dev = io or q.dtype, q.device
    if dt not in _IO:
        raise TypeError(f"unsupported io dtype {dt} (bf16 or fp32)")
    if dev.type != "cuda":
        raise ValueError("inputs must be on a HIP device")
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q must be [B, T, H, K] and v [B, T, HV, V]")
    B, T, H, K = q.shape
    HV, V = v.shape[2], v.shape[3]
    rows = q.dtype
    _check(q, "q", rows, (B, T, H, K), dev)
    _check(k, "k", rows, (B, T, H, K), dev)
    _check(v, "v", rows, (B, T, HV, V), dev)
    _check(g, "g", dt, (B, T, HV), dev)
    _check(beta, "beta", dt, (B, T, HV), dev)
    N, cu, h0 = B, None, None
    if cu_seqlens is not None:
        if cu_seqlens.dtype != torch.int64 or cu_seqlens.device != dev or cu_seqlens.dim() != 1:
            raise ValueError("cu_seqlens must be a 1-D int64 tensor on the inputs' device")
        if not cu_seqlens.is_contiguous():
            raise ValueError("cu_seqlens must be contiguous")
        N, cu = cu_seqlens.numel() - 1, cu_seqlens.data_ptr()
    if initial_state is not None:
        _check(initial_state, "initial_state", torch.float32, (N, HV, K, V), dev)
        h0 = initial_state.data_ptr()
    if gate not in _GATES:
        raise ValueError(f"gate must be None, 'softplus' or 'bounded' (got {gate!r})")
    A = bias = None
    if gate is not None:
        if A_log is None:
            raise ValueError("a gate needs A_log")
        _check(A_log, "A_log", torch.float32, (HV,), dev)
        A = A_log.data_ptr()
        if dt_bias is not None:
            _check(dt_bias, "dt_bias", torch.float32, (HV,), dev)
            bias = dt_bias.data_ptr()
    return GdnArgs(B, T, N, H, HV, K, V, _IO[dt], q.data_ptr(), k.data_ptr(), v.data_ptr(),
                   g.data_ptr(), beta.data_ptr(), float("nan") if scale is None else float(scale),
                   cu, h0, None, None, int(bool(use_qk_l2norm)), int(bool(use_beta_sigmoid)),
                   _GATES[gate], float(gate_lower_bound), A, bias)


def _aligned(*tensors):
    """The tensors, copied where they do not begin at a multiple of 16 bytes as the C ABI asks (g and beta of some
    tokens of a longer batch, for a call that reads them once)."""
    return (x if x.data_ptr() % 16 == 0 else x.clone() for x in tensors)


class GdnFwdPlan:
    """Validated arguments for repeated gdn_fwd calls on the same tensors.

    q, k [B,T,H,K]; v [B,T,HV,V]; g, beta [B,T,HV] (all bf16 or all fp32, contiguous, on one HIP
    device): g is the log decay of a token's whole state. cu_seqlens, initial_state, the outputs
    o and final_state and the pre-stage keywords are KdaFwdPlan's, with dt_bias fp32 [HV]. K and
    V are 64 or 128; any length, zero included. A plan's tensors begin at multiples of 16 bytes.
    final_state errs by about 4e-6 of itself for bf16 inputs, by 3e-7 where they are passed as fp32.
    """

    def __init__(self, q, k, v, g, beta, scale=None, cu_seqlens=None, initial_state=None,
                 output_final_state=True, workspace=None, o=None, final_state=None,
                 use_qk_l2norm=False, use_beta_sigmoid=False, gate=None, A_log=None,
                 dt_bias=None, gate_lower_bound=-5.0):
        self.lib = load()
        a = _arguments(q, k, v, g, beta, scale, cu_seqlens, initial_state, use_qk_l2norm,
                       use_beta_sigmoid, gate, A_log, dt_bias, gate_lower_bound)
        dev = self.device = q.device
        self.o = torch.empty_like(v) if o is None else o
        if o is not None:
            _check(o, "o", v.dtype, v.shape, dev)
        a.o = self.o.data_ptr()
        self.final_state = None
        if output_final_state:
            shape = (a.N, a.HV, a.K, a.V)
            self.final_state = (torch.empty(shape, dtype=torch.float32, device=dev)
                                if final_state is None else final_state)
            if final_state is not None:
                _check(final_state, "final_state", torch.float32, shape, dev)
            a.final_state = self.final_state.data_ptr()
        self.args = a
        self._keep = (q, k, v, g, beta, cu_seqlens, initial_state, A_log, dt_bias)
        # 0: refused (the call says why), or the recurrence, which needs none
        need = _on(dev, self.lib.gdn_fwd_workspace_bytes, ctypes.byref(a))
        if workspace is None:
            workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
        else:
            _check(workspace, "workspace", torch.uint8, workspace.shape, dev)
            if workspace.numel() < need:
                raise ValueError(f"workspace too small: {workspace.numel()} < {need} bytes")
        self.workspace = workspace

    def __call__(self, stream=None):
        """Enqueue the forward on `stream` (default: torch's current stream)."""
        _call(self.lib.gdn_fwd, "gdn_fwd", self.device, stream, ctypes.byref(self.args),
              self.workspace.data_ptr(), self.workspace.numel())
        return self.o, self.final_state


def gdn_fwd(q, k, v, g, beta, scale=None, cu_seqlens=None, initial_state=None,
            output_final_state=True, workspace=None, **prestage):
    """Gated delta rule forward. Returns (o, final_state or None; rows of o behind the last packed
    sequence hold anything); see GdnFwdPlan for shapes and the pre-stage keywords (use_qk_l2norm,
    use_beta_sigmoid, gate, A_log, dt_bias, gate_lower_bound)."""
    g, beta = _aligned(g, beta)
    return GdnFwdPlan(q, k, v, g, beta, scale, cu_seqlens, initial_state, output_final_state,
                      workspace, **prestage)()


class GdnBwdPlan:
    """Validated arguments for repeated gdn_bwd calls: gradients of gdn_fwd with respect to q, k, v,
    g, beta, initial_state and (with a gate) A_log, dt_bias, from d_o (like v) and dht (fp32
    [N,HV,K,V] or None).

    Inputs and pre-stage keywords as for GdnFwdPlan; q, k and v may all be Packed8 checkpoints (of
    one dtype, the io dtype), which every call unpacks into the workspace. Outputs, allocated once
    and reused by every call(): dq, dk, dv, dg, dbeta in the io dtype, dh0 fp32
    [N,HV,K,V] (when want_dh0), dA_log and ddt_bias fp32 [HV] (with a gate).
    """

    def __init__(self, q, k, v, g, beta, d_o, dht=None, scale=None, cu_seqlens=None,
                 initial_state=None, want_dh0=True, workspace=None, use_qk_l2norm=False,
                 use_beta_sigmoid=False, gate=None, A_log=None, dt_bias=None,
                 gate_lower_bound=-5.0):
        self.lib = load()
        packed = [isinstance(x, Packed8) for x in (q, k, v)]
        io, scales = None, ()
        if all(packed):
            io = q.dtype
            if k.dtype != io or v.dtype != io:
                raise TypeError("checkpoints of q, k and v must stand for one dtype")
            for x, name in ((q, "q"), (k, "k"), (v, "v")):
                _check_packed(x, name, q.data.device)
            scales = tuple(x.scale.data_ptr() for x in (q, k, v))
            self._packed = (q, k, v)
            q, k, v = q.data, k.data, v.data
        elif any(packed):
            raise TypeError("q, k and v must all be checkpoints or none (unpack8 gives a tensor)")
        a = _arguments(q, k, v, g, beta, scale, cu_seqlens, initial_state, use_qk_l2norm,
                       use_beta_sigmoid, gate, A_log, dt_bias, gate_lower_bound, io)
        dev = self.device = q.device
        io = io or q.dtype
        self._fn, name = ((self.lib.gdn_bwd_packed, self.lib.gdn_bwd_packed_workspace_bytes) if scales else
                          (self.lib.gdn_bwd, self.lib.gdn_bwd_workspace_bytes))
        _check(d_o, "d_o", io, v.shape, dev)
        shape = (a.N, a.HV, a.K, a.V)
        if dht is not None:
            _check(dht, "dht", torch.float32, shape, dev)
        f32 = dict(dtype=torch.float32, device=dev)
        self.dq, self.dk, self.dv = (torch.empty_like(x, dtype=io) for x in (q, k, v))
        self.dg, self.dbeta = torch.empty_like(g), torch.empty_like(beta)
        self.dh0 = torch.empty(shape, **f32) if want_dh0 else None
        self.dA_log = torch.empty(a.HV, **f32) if gate is not None else None
        self.ddt_bias = torch.empty(a.HV, **f32) if gate is not None else None
        self.args = a
        need = _on(dev, name, ctypes.byref(a))
        if need == 0 and a.B * a.T > 0:
            raise ValueError("unsupported shapes (K, V in {64, 128}; HV % H == 0)")
        if workspace is None:
            workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
        else:
            _check(workspace, "workspace", torch.uint8, workspace.shape, dev)
            if workspace.numel() < need:
                raise ValueError(f"workspace too small: {workspace.numel()} < {need} bytes")
        self.workspace = workspace
        outs = (self.dq, self.dk, self.dv, self.dg, self.dbeta, self.dh0, self.dA_log, self.ddt_bias)
        self._outs = outs
        self._ptrs = (ctypes.byref(a), *scales, _ptr(d_o), _ptr(dht), workspace.data_ptr(),
                      workspace.numel(), *map(_ptr, outs))
        self._keep = (q, k, v, g, beta, d_o, dht, cu_seqlens, initial_state, A_log, dt_bias)

    def __call__(self, stream=None):
        """Enqueue the backward on `stream` (default: torch's current stream); returns
        (dq, dk, dv, dg, dbeta, dh0, dA_log, ddt_bias)."""
        _call(self._fn, "gdn_bwd", self.device, stream, *self._ptrs)
        return self._outs


def gdn_bwd(q, k, v, g, beta, d_o, dht=None, scale=None, cu_seqlens=None, initial_state=None,
            want_dh0=True, **prestage):
    """Gated delta rule backward. Returns (dq, dk, dv, dg, dbeta in the io dtype, dh0 fp32 or None,
    dA_log or None, ddt_bias or None; rows behind the last packed sequence hold anything); see
    GdnBwdPlan. q, k and v may each be a Packed8
    checkpoint: the gradients are then those at the values that it stands for."""
    packed = [isinstance(x, Packed8) for x in (q, k, v)]
    if not all(packed):
        q, k, v = (unpack8(x) if p else x for x, p in zip((q, k, v), packed))
    g, beta = _aligned(g, beta)
    return GdnBwdPlan(q, k, v, g, beta, d_o, dht, scale, cu_seqlens, initial_state, want_dh0,
                      **prestage)()


class GdnStepPlan:
    """Validated arguments for repeated gdn_step calls on the same tensors (a serving loop that
    writes each step's inputs in place).

    q, k [B,T,H,K]; v [B,T,HV,V]; g, beta [B,T,HV]: T new tokens of B rows; state fp32
    [slots,HV,K,V], updated in place; state_indices int32 [B] on the device, or None for slot b
    of row b. A row whose index is negative or >= slots is padding: zeros in o, no state touched.
    Indices of other rows must differ. o [B,T,HV,V] is allocated once and reused. A plan's tensors begin
    at multiples of 16 bytes.
    """

    def __init__(self, q, k, v, g, beta, state, state_indices=None, scale=None, o=None,
                 use_qk_l2norm=False, use_beta_sigmoid=False, gate=None, A_log=None,
                 dt_bias=None, gate_lower_bound=-5.0):
        self.lib = load()
        a = _arguments(q, k, v, g, beta, scale, None, None, use_qk_l2norm, use_beta_sigmoid, gate,
                       A_log, dt_bias, gate_lower_bound)
        self.device = q.device
        _check(state, "state", torch.float32, (state.shape[0], a.HV, a.K, a.V), q.device)
        if state_indices is not None:
            _check(state_indices, "state_indices", torch.int32, (a.B,), q.device)
        elif state.shape[0] < a.B:
            raise ValueError(f"state has {state.shape[0]} slots for {a.B} rows")
        self.o = torch.empty_like(v) if o is None else o
        if o is not None:
            _check(o, "o", v.dtype, v.shape, q.device)
        a.o = self.o.data_ptr()
        self.args = a
        self._call = (ctypes.byref(a), state.data_ptr(), _ptr(state_indices), state.shape[0])
        self._keep = (q, k, v, g, beta, state, state_indices, A_log, dt_bias)

    def __call__(self, stream=None):
        """Enqueue the step on `stream` (default: torch's current stream)."""
        _call(self.lib.gdn_step, "gdn_step", self.device, stream, *self._call)
        return self.o


def gdn_step(q, k, v, g, beta, state, state_indices=None, scale=None, **prestage):
    """A serving step of the gated delta rule: returns o and updates `state` in place; see
    GdnStepPlan."""
    g, beta = _aligned(g, beta)
    return GdnStepPlan(q, k, v, g, beta, state, state_indices, scale, **prestage)()
