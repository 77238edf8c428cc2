"""Seeded inputs and error bars shared by the gated delta rule's tests.

Bars. o of bf16 io is rounded once, by at most half a step, 2^-8 of the value. What precedes the
rounding takes operands of two bf16 parts: a part pair holds x to 2^-17, and a product leaves out
the low-by-low term, at most another 2^-16 of its terms (2^-8 squared). Five products of that
kind follow each other from the inputs to o and to the state (K S, A R, then Q S and M e or
K^T e, with S itself such a sum), so an element errs by at most about 5 (2^-17 + 2^-16) = 1.1e-4
of the magnitudes that it sums. The tests hold elements to 2^-8 |ref| + 2^-11 rms and states
to 2^-13 relative L2 (errors of either sign average, which leaves a factor of ten).

fp32 io takes three parts (24 bits and dropped terms of 2^-24), so there the fp32 sums rule. A sum
of n terms rounds n times, each by at most 2^-24 of the partial sum. On the mean, with signs of
either kind, that is 2^-24 sqrt(n / 6) of the result: n = 128 and five sums one behind the other
give 2^-24 x 4.6 x sqrt(5) = 6e-7, and (I + L)^-1 may enlarge an error a few times over: 2^-18
(3.8e-6) relative L2, for o and for states. A single element has no such mean: every rounding may
have one sign, n 2^-24 = 2^-17 of the largest partial sum, which for random terms stays within
four times their rms: 2^-15 rms.
"""
from __future__ import annotations

import torch

STATE_TOL = {torch.bfloat16: 2.0 ** -13, torch.float32: 2.0 ** -18}
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
O_TOL = {torch.bfloat16: 2.0 ** -11, torch.float32: 2.0 ** -15}


def make(B=1, T=64, H=1, G=1, K=64, V=64, dtype=torch.bfloat16, lens=None, h0=False, raw=False,
         gate=None, dt_bias=True, seed=0, g_lo=0.9, g_hi=0.999, tail=0):
    """Keyword arguments of gdn_fwd (CPU tensors). lens: packed sequences; tail: tokens behind
    the last sequence."""
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)
    HV, N = H * G, B if lens is None else len(lens)
    cu = None
    if lens is not None:
        T = sum(lens) + tail
        cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int64)
    q, k, v, b = n(B, T, H, K), n(B, T, H, K), n(B, T, HV, V), n(B, T, HV)
    g = torch.log(g_lo + (g_hi - g_lo) * torch.rand(B, T, HV, generator=gen))
    if raw:
        q, k = 2 * q, 2 * k
    else:
        q, k = (x / (x.square().sum(-1, keepdim=True) + 1e-6).sqrt() for x in (q, k))
        b = torch.sigmoid(b)
    kw = {}
    if raw:
        kw.update(use_qk_l2norm=True, use_beta_sigmoid=True)
    if gate:
        g = n(B, T, HV) - 1
        kw.update(gate=gate, A_log=torch.log(0.5 + 1.5 * torch.rand(HV, generator=gen)),
                  dt_bias=0.5 * n(HV) if dt_bias else None)
    a = dict(q=q.to(dtype), k=k.to(dtype), v=v.to(dtype), g=g.to(dtype), beta=b.to(dtype))
    if cu is not None:
        a["cu_seqlens"] = cu
    if h0:
        a["initial_state"] = 0.3 * n(N, HV, K, V)
    return a | kw


def to(a, device):
    return {n: x.to(device) if torch.is_tensor(x) else x for n, x in a.items()}


def check_o(o, ref, dtype, rows=None):
    """Every element (rms over the compared rows of a head), and for fp32 the whole in L2."""
    o, ref = o.double().cpu(), ref.double()
    if rows is not None:
        o, ref = o[:, :rows], ref[:, :rows]
    assert torch.isfinite(o).all()
    rms = ref.square().mean(dim=(0, 1, 3), keepdim=True).sqrt()
    over = (o - ref).abs() - (ROUND[dtype] * ref.abs() + O_TOL[dtype] * rms)
    assert (over <= 0).all(), f"worst element {over.max():.3e} over its bound"
    if dtype == torch.float32:
        assert (o - ref).norm() <= 2.0 ** -18 * ref.norm()


def check_state(s, ref, dtype):
    s, ref = s.double().cpu(), ref.double()
    assert torch.isfinite(s).all()
    err = (s - ref).flatten(2).norm(dim=2)
    assert (err <= STATE_TOL[dtype] * ref.flatten(2).norm(dim=2)).all(), \
        f"worst state {(err / ref.flatten(2).norm(dim=2)).max():.3e}"
