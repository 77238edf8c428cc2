"""fp64 gated linear recurrence with one state a channel, by the token recurrence (test infrastructure, CPU):

    h <- e^{g_t} h + beta_t x_t;   y_t = h

and its gradients from their formulas, written out:

    dh_t = dy_t + m_{t+1};  m_t = e^{g_t} dh_t;  dx_t = beta_t dh_t;  dbeta_t = x_t dh_t;  dg_t = h_{t-1} m_t

with m = dht behind the last token and dh0 = m_0."""
from __future__ import annotations

import torch
import torch.nn.functional as F


def prestage(g, beta, use_beta_sigmoid=False, gate=None, A_log=None, dt_bias=None, gate_lower_bound=-5.0):
    if use_beta_sigmoid:
        beta = torch.sigmoid(beta)
    if gate is not None:
        u = g if dt_bias is None else g + dt_bias
        a = torch.exp(A_log)
        g = -a * F.softplus(u, threshold=1e9) if gate == "softplus" else gate_lower_bound * torch.sigmoid(a * u)
    return g, beta


def _spans(B, T, cu_seqlens):
    return [(b * T, b * T + T) for b in range(B)] if cu_seqlens is None else [
        (int(a), int(b)) for a, b in zip(cu_seqlens[:-1], cu_seqlens[1:])]


def glr_recurrent(x, g, beta=None, initial_state=None, cu_seqlens=None, **pre):
    """y [B,T,D] and the final states [N,D] in fp64; all arguments CPU tensors. Differentiable by autograd."""
    f = lambda t: t.double() if torch.is_tensor(t) else t
    g, beta = prestage(f(g), f(beta), **{n: f(t) for n, t in pre.items()})
    B, T, D = x.shape
    w = (f(x) if beta is None else beta * f(x)).reshape(B * T, D)
    a = torch.exp(g).reshape(B * T, D)
    spans = _spans(B, T, cu_seqlens)
    h0 = torch.zeros(len(spans), D, dtype=torch.float64) if initial_state is None else f(initial_state)
    y, fin = [], []
    for h, (lo, hi) in zip(h0, spans):
        for t in range(lo, hi):
            h = a[t] * h + w[t]
            y.append(h)
        fin.append(h)
    tail = torch.zeros(B * T - spans[-1][1], D, dtype=torch.float64)
    y = torch.cat([torch.stack(y), tail]) if y else tail
    return y.reshape(B, T, D), torch.stack(fin)


def glr_gradients(x, g, y, d_y, beta=None, dht=None, initial_state=None, cu_seqlens=None, **pre):
    """{name: fp64 gradient} by the formulas above, h_{t-1} read from y as given."""
    f = lambda t: t.double() if torch.is_tensor(t) else t
    pre = {n: f(t) for n, t in pre.items()}
    raw_g, raw_beta = f(g), f(beta)
    with torch.enable_grad():
        leaves = {"g": raw_g.clone().requires_grad_()}
        leaves |= {n: pre[n].clone().requires_grad_() for n in ("A_log", "dt_bias") if torch.is_tensor(pre.get(n))}
        g, beta = prestage(leaves["g"], raw_beta, **(pre | {n: t for n, t in leaves.items() if n != "g"}))
    B, T, D = d_y.shape
    a, dy, y = torch.exp(g.detach()).reshape(B * T, D), f(d_y).reshape(B * T, D), f(y).reshape(B * T, D)
    spans = _spans(B, T, cu_seqlens)
    h0 = torch.zeros(len(spans), D, dtype=torch.float64) if initial_state is None else f(initial_state)
    dh, dg = torch.zeros_like(dy), torch.zeros_like(dy)
    dh0 = torch.zeros_like(h0) if dht is None else f(dht).clone()
    for s, (lo, hi) in enumerate(spans):
        m = dh0[s].clone()
        for t in reversed(range(lo, hi)):
            dh[t] = dy[t] + m
            m = a[t] * dh[t]
            dg[t] = (y[t - 1] if t > lo else h0[s]) * m
        dh0[s] = m
    dh, dg = dh.reshape(B, T, D), dg.reshape(B, T, D)
    out = {"x": dh if beta is None else beta * dh, "initial_state": dh0, "dh": dh, "dg_active": dg}
    if beta is not None:
        out["beta"] = f(x) * dh * (beta * (1 - beta) if pre.get("use_beta_sigmoid") else 1)
    if pre.get("gate") is None:
        out["g"] = dg
    else:                                   # the gate's own derivative
        out |= dict(zip(leaves, torch.autograd.grad((g * dg).sum(), list(leaves.values()))))
    return out
