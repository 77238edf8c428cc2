"""Seeded inputs and error bounds shared by the tests of the gated linear recurrence.

Bounds are propagated with the recurrence itself. Token t adds a rounding error of at most c 2^-24 M_t to
the state, M the recurrence of magnitudes (M_t = a_t M_{t-1} + |w_t|), and earlier errors decay with the
state: B_t = a_t B_{t-1} + c 2^-24 M_t. What c counts, in units of 2^-24 of M_t: two fused steps (2), a decay
in its two-number form or as an exponential of up to one unit in the last place (2), beta's sigmoid and its
product with x (6: an exponential, a sum, a division or an approximate reciprocal, the product), and, once a
step of 64 tokens or more, products of up to 11 decays of groups and waves (22, of which one token has less than one).
A gate's log decay errs by a few units of itself, |g| e^g <= 1/e of them in a (4). So c = 16 for fp32 io; bf16
io takes base-2 exponentials of a rounded product with log2 e, |g| log2 e more units for a decay e^g <
e^-1/2, that is 2 |g| e^g <= 1, and sigmoids that err likewise: c = 32. A strong decay makes M_t small in the
same measure, but for its own error: |g| 2^-23 of a state that it has just made as small; the tests of strong
decays add it (`strong`).

A result in bf16 is rounded by up to 2^-8 of itself more, in fp32 by 2^-24.
"""
from __future__ import annotations

import torch

from oracle.glr import prestage

ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
STEPS = {torch.bfloat16: 32 * 2.0 ** -24, torch.float32: 16 * 2.0 ** -24}


def make(B=1, T=64, D=64, dtype=torch.bfloat16, lens=None, h0=False, beta=False, sigmoid=False, gate=None,
         dt_bias=True, seed=0, g_lo=0.9, g_hi=0.999, tail=0):
    """Keyword arguments of glr_fwd (CPU tensors). lens: packed sequences; tail: tokens behind the last."""
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)
    N, cu = B if lens is None else len(lens), None
    if lens is not None:
        T = sum(lens) + tail
        cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int64)
    a = {"x": n(B, T, D).to(dtype)}
    a["g"] = (n(B, T, D) - 1 if gate else torch.log(g_lo + (g_hi - g_lo) * torch.rand(B, T, D, generator=gen))).to(dtype)
    if beta or sigmoid:
        b = n(B, T, D)
        a["beta"] = (b if sigmoid else torch.sigmoid(b)).to(dtype)
    if sigmoid:
        a["use_beta_sigmoid"] = True
    if gate:
        a |= dict(gate=gate, A_log=torch.log(0.5 + 1.5 * torch.rand(D, generator=gen)), dt_bias=0.5 * n(D) if dt_bias else None)
    if cu is not None:
        a["cu_seqlens"] = cu
    if h0:
        a["initial_state"] = n(N, D)
    return a


def to(a, device):
    return {n: x.to(device) if torch.is_tensor(x) else x for n, x in a.items()}


def spans_of(a):
    B, T, _ = a["g"].shape
    cu = a.get("cu_seqlens")
    return [(b * T, b * T + T) for b in range(B)] if cu is None else [(int(p), int(q)) for p, q in zip(cu[:-1], cu[1:])]


def _scan_bound(a, w, start, spans, unit, reverse=False):
    """(B_t for every token, B behind every sequence) of the recurrence with decays a and inputs w."""
    out, ends = torch.zeros_like(w), torch.zeros_like(start)
    mags = torch.zeros_like(w)
    for s, (lo, hi) in enumerate(spans):
        M, b = start[s].abs(), torch.zeros_like(start[s])
        for t in reversed(range(lo, hi)) if reverse else range(lo, hi):
            if reverse:                     # dh = dy + m; m = a dh
                M = w[t].abs() + M
                b = b + unit * M
                out[t], mags[t] = b, M
                M, b = a[t] * M, a[t] * b + unit * a[t] * M
            else:
                M = a[t] * M + w[t].abs()
                b = a[t] * b + unit * M
                out[t], mags[t] = b, M
        ends[s] = b
    return out, ends, mags


def _active(a):
    f = lambda t: t.double() if torch.is_tensor(t) else t
    pre = {n: f(a[n]) for n in ("use_beta_sigmoid", "gate", "A_log", "dt_bias", "gate_lower_bound") if n in a}
    return prestage(f(a["g"]), f(a.get("beta")), **pre)


def forward_bound(a):
    """Bounds of y's (before its rounding) and the final states' errors."""
    g, beta = _active(a)
    B, T, D = g.shape
    w = a["x"].double() if beta is None else beta * a["x"].double()
    spans = spans_of(a)
    h0 = a["initial_state"].double() if "initial_state" in a else torch.zeros(len(spans), D, dtype=torch.float64)
    out, ends, _ = _scan_bound(torch.exp(g).reshape(-1, D), w.reshape(-1, D), h0, spans, STEPS[a["x"].dtype])
    return out.reshape(B, T, D), ends


def check(got, ref, bound, dtype, what):
    got, ref = got.double().cpu(), ref.double()
    assert got.shape == ref.shape, what
    assert torch.isfinite(got).all(), what
    over = (got - ref).abs() - (ROUND[dtype] * (ref.abs() + bound) + bound)
    assert got.numel() == 0 or (over <= 0).all(), f"{what}: worst element {over.max():.3e} over its bound"


def check_forward(a, y, fin, ref_y, ref_fin):
    by, bf = forward_bound(a)
    rows = spans_of(a)[-1][1] if "cu_seqlens" in a else y.shape[1]
    check(y[:, :rows], ref_y[:, :rows], by[:, :rows], y.dtype, "y")
    if fin is not None:
        check(fin, ref_fin, bf, torch.float32, "final_state")


def check_gradients(a, y, d_y, dht, got, ref):
    """got: (dx, dg, dbeta, dh0, dA_log, ddt_bias) against glr_gradients' formulas at the same y."""
    dtype, unit = a["x"].dtype, STEPS[a["x"].dtype]
    g, beta = _active(a)
    B, T, D = g.shape
    spans = spans_of(a)
    flat = lambda t: t.double().reshape(-1, D)
    e = torch.exp(flat(g))
    start = torch.zeros(len(spans), D, dtype=torch.float64) if dht is None else dht.double()
    bd, bend, mag = _scan_bound(e, flat(d_y), start, spans, unit, reverse=True)
    before = torch.zeros_like(e)
    for s, (lo, hi) in enumerate(spans):
        if hi > lo:
            before[lo] = a["initial_state"][s].double() if "initial_state" in a else 0.0
            before[lo + 1:hi] = flat(y)[lo:hi - 1]
    b = torch.ones_like(e) if beta is None else flat(beta)
    rows = spans[-1][1]
    cut = lambda t: t.reshape(-1, D)[:rows]
    dx, dg, dbeta, dh0, dA, db = got
    check(cut(dx), cut(ref["x"]), cut(b.abs() * (bd + unit * mag)), dtype, "dx")
    # the active decay's gradient, and a gate's derivative on top: a handful of roundings more
    bg = before.abs() * (e * bd + unit * e * mag)
    if "gate" in a:
        u = flat(a["g"]) + (0.0 if a.get("dt_bias") is None else a["dt_bias"].double())
        A = torch.exp(a["A_log"].double())
        lb = a.get("gate_lower_bound", -5.0)
        if a["gate"] == "softplus":
            slope, dact = A * torch.sigmoid(u), flat(g).abs()
        else:
            r = torch.sigmoid(A * u)
            slope, dact = abs(lb) * r * (1 - r) * A, abs(lb) * r * (1 - r) * (A * u).abs()
        # a sigmoid of z, and its derivative, err by |z| 2^-23 of themselves besides a few roundings
        part = (2 + (A * u).abs()) * unit * before.abs() * e * mag
        bu = slope * (bg + part)
        check(cut(dg), cut(ref["g"]), cut(bu), dtype, "dg")
        ba = dact * (bg + part)
        check(dA, ref["A_log"], ba[:rows].sum(0), torch.float32, "dA_log")
        if a.get("dt_bias") is not None:
            check(db, ref["dt_bias"], bu[:rows].sum(0), torch.float32, "ddt_bias")
    else:
        check(cut(dg), cut(ref["g"]), cut(bg), dtype, "dg")
        assert dA is None and db is None
    if beta is not None:
        x = flat(a["x"]).abs()
        bb = x * (bd + unit * mag)
        if a.get("use_beta_sigmoid"):
            bb = (bb + (2 + flat(a["beta"]).abs()) * unit * x * mag) * b * (1 - b)
        check(cut(dbeta), cut(ref["beta"]), cut(bb), dtype, "dbeta")
    else:
        assert dbeta is None
    if dh0 is not None:
        check(dh0, ref["initial_state"], bend, torch.float32, "dh0")
