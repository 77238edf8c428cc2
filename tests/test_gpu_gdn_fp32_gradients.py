"""fp32 gradients of the gated delta rule on the inputs that are hardest for them, against autograd through
the fp64 token recurrence: decays of any strength next to mild ones, keys that resemble each other (whose
powers of L grow while the inverse stays of size one), cleared states, long and ragged sequences. The bar is
the fp32 one of the other gradient tests, 2^-16 relative L2: fp32 sums behind each other, and inverses formed
by substitution, which lose no digits to the powers of L."""
from __future__ import annotations

import pytest
import torch

import chunked_kimi_delta_amd as kda
from gdn_cases import make, to
from oracle.gdn import gdn_gradients
from test_gpu_gdn_backward import LEAVES, OUTS, compare, cotangents

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
FP = torch.float32


def check(a):
    d_o, dh = cotangents(a)
    got = dict(zip(OUTS, kda.gdn_bwd(**to(a, DEV), d_o=d_o.to(DEV), dht=dh.to(DEV),
                                     want_dh0="initial_state" in a)))
    leaves = {n: a[n] for n in LEAVES if a.get(n) is not None}
    ref = gdn_gradients(leaves, d_o, dh, **{n: x for n, x in a.items() if n not in LEAVES})
    # fp32 has its 24 bits from 2^-126 up: what 64 bits hold below (e^-100, e^-600) is not compared
    normal = lambda d: {n: torch.where(x.abs() < 2.0 ** -126, 0.0, x) for n, x in d.items() if x is not None}
    compare(normal(got), normal(ref), FP)


@pytest.mark.parametrize("K,V", [(64, 64), (128, 128)])
@pytest.mark.parametrize("kind", ["strong", "mixed", "none", "bursts", "clears"])
def test_decays(kind, K, V):
    a = make(T=150, H=2, K=K, V=V, h0=True, seed=3, dtype=FP)
    g = a["g"]
    if kind == "strong":
        g.mul_(0).sub_(40.0)
    elif kind == "mixed":           # one huge decay, then slow ones
        g[:, 5] = -3000.0
    elif kind == "bursts":          # some strong ones, then slow ones among the same few tokens
        for t in range(0, 150, 16):
            g[:, t:t + 6] = -100.0
    elif kind == "clears":
        g[:, 2::37] = -torch.inf
    else:
        g.zero_()
    check(a)


def decayed_states(a, d_o, dh):
    """By token and head in fp64: the norms of the state behind its decay and of the loss's gradient by that state."""
    q, k, v, g, beta = (a[n][0].double() for n in ("q", "k", "v", "g", "beta"))
    S, bumps, norms, loss = torch.zeros(dh.shape[1:], dtype=torch.float64), [], [], 0.0
    for t in range(len(q)):
        bumps.append(torch.zeros_like(S, requires_grad=True))
        S = torch.exp(g[t])[:, None, None] * S + bumps[-1]
        norms.append(S.detach().flatten(1).norm(dim=1))
        r = v[t] - (S * k[t][:, :, None]).sum(1)
        S = S + (beta[t][:, None] * k[t])[:, :, None] * r[:, None, :]
        loss = loss + (k.shape[-1] ** -0.5 * (S * q[t][:, :, None]).sum(1) * d_o[0, t].double()).sum()
    grads = torch.autograd.grad(loss + (S * dh[0].double()).sum(), bumps)
    return torch.stack(norms), torch.stack([x.flatten(1).norm(dim=1) for x in grads])


@pytest.mark.parametrize("spread", [0.0, 0.02, 0.1])
def test_keys_that_resemble_each_other(spread):
    a = make(T=130, H=2, K=64, V=64, seed=4, dtype=FP)
    gen = torch.Generator().manual_seed(11)
    k = a["k"][:, :1] + spread * a["k"]
    a["k"] = k / k.norm(dim=-1, keepdim=True)
    a["beta"] = 0.9 + 0.1 * torch.rand(a["beta"].shape, generator=gen)
    a["g"] = torch.full_like(a["g"], -0.005)
    d_o, dh = cotangents(a)
    got = dict(zip(OUTS, kda.gdn_bwd(**to(a, DEV), d_o=d_o.to(DEV), dht=dh.to(DEV), want_dh0=False)))
    ref = gdn_gradients({n: a[n] for n in LEAVES if n in a}, d_o, dh)
    # dg_t = <S, dS> of the state behind the decay and its gradient. With errors dS' and S' of 2^-16 each it is off
    # by |<S', dS> + <S, dS'>| <= 2 x 2^-16 |S| |dS|. Where all keys are one, dg is some millionths of |S| |dS|
    # (each write takes back what the decay left, so the gradient hardly meets the state), and plain fp32 steps
    # of the recurrence give 1.2e-4 relative to it; there that bound alone is held.
    S, dS = decayed_states(a, d_o, dh)
    assert ((got["g"][0].double().cpu() - ref["g"][0]).abs() <= 2.0 ** -15 * S * dS).all()
    if spread == 0.0:
        del ref["g"]
    compare(got, ref, FP)


def test_a_cleared_state_passes_no_gradient_at_all():
    # at g = -inf the state starts anew: nothing before it sees what follows, in dg either
    a = make(T=100, H=1, K=64, V=64, dtype=FP, h0=True)
    a["g"][:, 70] = -torch.inf
    d_o, dh = cotangents(a)
    d_o[:, :70] = 0
    out = dict(zip(OUTS, kda.gdn_bwd(**to(a, DEV), d_o=d_o.to(DEV), dht=dh.to(DEV))))
    for n in ("q", "k", "v", "g", "beta"):
        assert (out[n][:, :70] == 0).all(), n
    assert (out["g"][:, 70] == 0).all() and (out["initial_state"] == 0).all()
    compare(out, gdn_gradients({n: a[n] for n in LEAVES if n in a}, d_o, dh), FP)


@pytest.mark.parametrize("kw", [
    dict(T=1030, G=1, K=128, V=128), dict(lens=[900, 0, 64, 600, 1], G=2, K=64, V=64, raw=True, gate="bounded")])
def test_long(kw):
    check(make(H=1, h0=True, dtype=FP, **kw))
