"""torch.autograd integration: chunk_kda runs kda_fwd forward and kda_bwd backward (argument
marshalling only; both directions are the library's kernels)."""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from .act8 import Packed8, pack8, unpack8
from .api import _zero_tail, kda_bwd, kda_fwd
from .gdn import GdnBwdPlan, GdnFwdPlan, _aligned
from .glr import GlrBwdPlan, GlrFwdPlan


def _save(ctx, checkpoint, q, k, v, *rest):
    """Keep a forward's tensors for its backward; with checkpoint "int8", q, k and v as Packed8."""
    if checkpoint not in (None, "int8"):
        raise ValueError(f"checkpoint must be None or 'int8' (got {checkpoint!r})")
    ctx.packed = checkpoint is not None
    if ctx.packed:
        p = [pack8(x) for x in (q, k, v)]
        ctx.save_for_backward(*(x.data for x in p), *(x.scale for x in p), *rest)
        ctx.dtypes = [x.dtype for x in p]
    else:
        ctx.save_for_backward(q, k, v, *rest)


def _saved(ctx):
    """(q, k, v as kept: tensors or Packed8, then the rest)."""
    t = ctx.saved_tensors
    if not ctx.packed:
        return t
    return tuple(Packed8(*x) for x in zip(t[:3], t[3:6], ctx.dtypes)) + t[6:]


class ChunkKDAFunction(torch.autograd.Function):
    """o, final_state = KDA(q, k, v, g, beta; initial_state), differentiable (once) in q, k, v, g, beta,
    initial_state and (with a gate) A_log, dt_bias. Gradients come back in the dtype of each
    input (the kernels compute them in fp32)."""

    @staticmethod
    def forward(ctx, q, k, v, g, beta, initial_state, A_log, dt_bias, scale, cu_seqlens,
                use_qk_l2norm, use_beta_sigmoid, gate, gate_lower_bound, checkpoint=None):
        pre = dict(use_qk_l2norm=use_qk_l2norm, use_beta_sigmoid=use_beta_sigmoid, gate=gate,
                   A_log=A_log, dt_bias=dt_bias, gate_lower_bound=gate_lower_bound)
        o, fin = kda_fwd(q, k, v, g, beta, scale=scale, cu_seqlens=cu_seqlens,
                         initial_state=initial_state, output_final_state=True, **pre)
        _zero_tail(cu_seqlens, o)           # the kernels leave rows behind the last sequence alone
        _save(ctx, checkpoint, q, k, v, g, beta, initial_state, A_log, dt_bias, cu_seqlens)
        ctx.scale = scale
        ctx.pre = dict(use_qk_l2norm=use_qk_l2norm, use_beta_sigmoid=use_beta_sigmoid, gate=gate,
                       gate_lower_bound=gate_lower_bound)
        return o, fin

    @staticmethod
    @once_differentiable
    def backward(ctx, d_o, d_fin):
        q, k, v, g, beta, h0, A_log, dt_bias, cu = _saved(ctx)
        if ctx.packed:
            q, k, v = unpack8(q), unpack8(k), unpack8(v)
        d_o = (torch.zeros_like(v) if d_o is None else d_o.to(v.dtype)).contiguous()
        dht = None if d_fin is None else d_fin.float().contiguous()
        dq, dk, dv, dg, db, dh0, dA, ddt = kda_bwd(
            q, k, v, g, beta, d_o, dht, scale=ctx.scale, cu_seqlens=cu, initial_state=h0,
            want_dh0=h0 is not None, A_log=A_log, dt_bias=dt_bias, **ctx.pre)
        _zero_tail(cu, dq, dk, dv, dg, db)
        cast = lambda x, ref: None if x is None or ref is None else x.to(ref.dtype)
        return (cast(dq, q), cast(dk, k), cast(dv, v), cast(dg, g), cast(db, beta),
                cast(dh0, h0), cast(dA, A_log), cast(ddt, dt_bias),
                None, None, None, None, None, None, None)


def chunk_kda(q, k, v, g, beta, scale=None, initial_state=None, cu_seqlens=None,
              use_qk_l2norm=False, use_beta_sigmoid=False, gate=None, A_log=None, dt_bias=None,
              gate_lower_bound=-5.0, checkpoint=None):
    """Differentiable KDA forward; returns (o, final_state). Shapes as KdaFwdPlan; every
    tensor argument may require grad (cu_seqlens excepted). The forward uses the library's
    default chunk; the backward always uses 16-token chunks. checkpoint="int8" keeps q, k and v
    for the backward in 8 bits (pack8), which then gives the gradients at those values. Rows behind the
    last packed sequence are zero in o and in the gradients."""
    return ChunkKDAFunction.apply(q, k, v, g, beta, initial_state, A_log, dt_bias, scale,
                                  cu_seqlens, use_qk_l2norm, use_beta_sigmoid, gate,
                                  gate_lower_bound, checkpoint)


class ChunkGDNFunction(torch.autograd.Function):
    """o, final_state = gated delta rule(q, k, v, g, beta; initial_state), differentiable (once) as
    ChunkKDAFunction is."""

    @staticmethod
    def forward(ctx, q, k, v, g, beta, initial_state, A_log, dt_bias, scale, cu_seqlens,
                use_qk_l2norm, use_beta_sigmoid, gate, gate_lower_bound, checkpoint=None):
        ctx.pre = dict(use_qk_l2norm=use_qk_l2norm, use_beta_sigmoid=use_beta_sigmoid, gate=gate,
                       gate_lower_bound=gate_lower_bound)
        g, beta = _aligned(g, beta)
        plan = GdnFwdPlan(q, k, v, g, beta, scale=scale, cu_seqlens=cu_seqlens,
                          initial_state=initial_state, A_log=A_log, dt_bias=dt_bias, **ctx.pre)
        o, fin = plan()
        _zero_tail(cu_seqlens, o)
        _save(ctx, checkpoint, q, k, v, g, beta, initial_state, A_log, dt_bias, cu_seqlens)
        ctx.scale = scale
        return o, fin

    @staticmethod
    @once_differentiable
    def backward(ctx, d_o, d_fin):
        q, k, v, g, beta, h0, A_log, dt_bias, cu = _saved(ctx)
        d_o = d_o.to(g.dtype).contiguous()
        plan = GdnBwdPlan(
            q, k, v, g, beta, d_o, d_fin.float().contiguous(), scale=ctx.scale, cu_seqlens=cu,
            initial_state=h0, want_dh0=h0 is not None, A_log=A_log, dt_bias=dt_bias, **ctx.pre)
        dq, dk, dv, dg, db, dh0, dA, ddt = plan()
        _zero_tail(cu, dq, dk, dv, dg, db)
        return (dq, dk, dv, dg, db, dh0, dA, None if dt_bias is None else ddt,
                None, None, None, None, None, None, None)


def chunk_gdn(q, k, v, g, beta, scale=None, initial_state=None, cu_seqlens=None,
              use_qk_l2norm=False, use_beta_sigmoid=False, gate=None, A_log=None, dt_bias=None,
              gate_lower_bound=-5.0, checkpoint=None):
    """Differentiable gated delta rule (one decay per token and value head); returns (o,
    final_state). Shapes as GdnFwdPlan; every tensor argument may require grad (cu_seqlens
    excepted). checkpoint="int8" keeps q, k and v for the backward in 8 bits (pack8), which then
    gives the gradients at those values. Rows behind the last packed sequence are zero in o and in
    the gradients."""
    return ChunkGDNFunction.apply(q, k, v, g, beta, initial_state, A_log, dt_bias, scale,
                                  cu_seqlens, use_qk_l2norm, use_beta_sigmoid, gate,
                                  gate_lower_bound, checkpoint)


class ChunkGLRFunction(torch.autograd.Function):
    """y, final_state = gated linear recurrence(x, g, beta; initial_state), differentiable (once) in every
    tensor argument but cu_seqlens."""

    @staticmethod
    def forward(ctx, x, g, beta, initial_state, A_log, dt_bias, cu_seqlens, use_beta_sigmoid, gate,
                gate_lower_bound):
        ctx.pre = dict(use_beta_sigmoid=use_beta_sigmoid, gate=gate, gate_lower_bound=gate_lower_bound)
        y, fin = GlrFwdPlan(x, g, beta, cu_seqlens, initial_state, A_log=A_log, dt_bias=dt_bias, **ctx.pre)()
        _zero_tail(cu_seqlens, y)
        ctx.save_for_backward(None if beta is None else x, g, beta, initial_state, A_log, dt_bias, cu_seqlens, y)
        return y, fin

    @staticmethod
    @once_differentiable
    def backward(ctx, d_y, d_fin):
        x, g, beta, h0, A_log, dt_bias, cu, y = ctx.saved_tensors
        plan = GlrBwdPlan(x, g, y, d_y.to(g.dtype).contiguous(), beta, d_fin.float().contiguous(), cu, h0,
                          want_dh0=h0 is not None, A_log=A_log, dt_bias=dt_bias, **ctx.pre)
        dx, dg, db, dh0, dA, ddt = plan()
        _zero_tail(cu, dx, dg, *(() if db is None else (db,)))
        return dx, dg, db, dh0, dA, None if dt_bias is None else ddt, None, None, None, None


def chunk_glr(x, g, beta=None, initial_state=None, cu_seqlens=None, use_beta_sigmoid=False, gate=None, A_log=None,
              dt_bias=None, gate_lower_bound=-5.0):
    """Differentiable gated linear recurrence (one state a channel); returns (y, final_state). Shapes as
    GlrFwdPlan; every tensor argument may require grad (cu_seqlens excepted). The backward takes the states from
    y, which must not be changed in place before it. Rows behind the last packed sequence are zero in y and in the
    gradients."""
    return ChunkGLRFunction.apply(x, g, beta, initial_state, A_log, dt_bias, cu_seqlens, use_beta_sigmoid, gate,
                                  gate_lower_bound)
