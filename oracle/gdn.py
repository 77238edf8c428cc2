"""fp64 gated delta rule with one decay per token and value head, by the token recurrence (test
infrastructure, CPU):

    S <- e^{g_t} S;   r = v_t - S^T k_t;   S <- S + beta_t k_t r^T;   o_t = scale S^T q_t

per sequence and value head j, with q/k head j / (HV / H). Written with torch fp64 ops that
autograd differentiates, so the gradients are those of these four lines and of the pre-stage
(q/k L2 norm, beta sigmoid, gate activation) as given below."""
from __future__ import annotations

import torch
import torch.nn.functional as F


def prestage(q, k, g, beta, use_qk_l2norm=False, use_beta_sigmoid=False, gate=None, A_log=None,
             dt_bias=None, gate_lower_bound=-5.0):
    if use_qk_l2norm:
        q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + 1e-6)
        k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + 1e-6)
    if use_beta_sigmoid:
        beta = torch.sigmoid(beta)
    if gate is not None:
        x = g if dt_bias is None else g + dt_bias
        a = torch.exp(A_log)
        g = -a * F.softplus(x, threshold=1e9) if gate == "softplus" else gate_lower_bound * torch.sigmoid(a * x)
    return q, k, g, beta


def gdn_recurrent(q, k, v, g, beta, scale=None, initial_state=None, cu_seqlens=None, **pre):
    """o [B,T,HV,V] and the final states [N,HV,K,V] in fp64; all arguments CPU tensors."""
    f = lambda x: None if x is None else x.double()
    pre = {n: f(x) if torch.is_tensor(x) else x for n, x in pre.items()}
    q, k, g, beta = prestage(f(q), f(k), f(g), f(beta), **pre)
    v, h0 = f(v), f(initial_state)
    B, T, H, K = q.shape
    HV, V = v.shape[2:]
    q, k = (x.repeat_interleave(HV // H, 2).reshape(B * T, HV, K) for x in (q, k))
    v, g, beta = v.reshape(B * T, HV, V), g.reshape(B * T, HV), beta.reshape(B * T, HV)
    cu = ([b * T for b in range(B + 1)] if cu_seqlens is None else [int(x) for x in cu_seqlens])
    scale = K ** -0.5 if scale is None else scale
    o, fin = [], []
    for s in range(len(cu) - 1):
        S = torch.zeros(HV, K, V, dtype=torch.float64) if h0 is None else h0[s]
        for t in range(cu[s], cu[s + 1]):
            S = torch.exp(g[t])[:, None, None] * S
            r = v[t] - (S * k[t][:, :, None]).sum(1)
            S = S + (beta[t][:, None] * k[t])[:, :, None] * r[:, None, :]
            o.append(scale * (S * q[t][:, :, None]).sum(1))
        fin.append(S)
    rows = cu[-1]
    out = torch.zeros(B * T, HV, V, dtype=torch.float64)
    if o:
        out = torch.cat([torch.stack(o), out[rows:]])
    return out.reshape(B, T, HV, V), torch.stack(fin)


def gdn_gradients(inputs, d_o, dht=None, **kw):
    """{name: fp64 gradient} of sum(o d_o) + sum(final dht) for every tensor of `inputs` (a dict
    of gdn_recurrent's differentiable arguments: q, k, v, g, beta, initial_state, A_log,
    dt_bias)."""
    leaves = {n: x.double().clone().requires_grad_() for n, x in inputs.items() if x is not None}
    o, fin = gdn_recurrent(**leaves, **kw)
    loss = (o * d_o.double()).sum()
    if dht is not None:
        loss = loss + (fin * dht.double()).sum()
    grads = torch.autograd.grad(loss, list(leaves.values()), allow_unused=True)
    return {n: torch.zeros_like(x) if d is None else d for (n, x), d in zip(leaves.items(), grads)}
