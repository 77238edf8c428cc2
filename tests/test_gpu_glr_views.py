"""Inputs of the gated linear recurrence that are some tokens of a longer batch, on the GPU: the bits of their copies, and
nothing of what lies around them."""
from __future__ import annotations

import pytest
import torch

import chunked_kimi_delta_amd as kda
from glr_cases import check_forward, check_gradients, make, to
from oracle.glr import glr_gradients, glr_recurrent

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = [torch.bfloat16, torch.float32]


def inside(t, ahead, behind, columns=0):
    """t as tokens (and columns) of a longer batch, NaN elsewhere."""
    B, T, D = t.shape
    wide = torch.full((B, ahead + T + behind, D + columns), float("nan"), dtype=t.dtype, device=t.device)
    view = wide[:, ahead:ahead + T, columns:]
    view.copy_(t)
    return view


def same(got, want):
    for p, q in zip(got, want):
        assert (p is None and q is None) or torch.equal(p, q)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pre", [dict(), dict(sigmoid=True, gate="softplus")], ids=["plain", "raw"])
@pytest.mark.parametrize("columns", [0, 6, 7])
@pytest.mark.parametrize("B,T,D", [(3, 40, 12), (2, 1, 33), (3, 5000, 66), (2, 700, 1300), (80, 9, 120)])
def test_tokens_of_a_longer_batch(B, T, D, columns, pre, dtype):
    """The bits of the copies. Not so where bf16 tiles take one channel a lane for rows that begin at odd elements, and two
    for the copies: a wave's decays all take one form (e^g or e^g - 1), which then other channels decide. Either form
    is within the bounds of the recurrence in 64 bits, and those hold there."""
    cpu = make(B=B, T=T, D=D, h0=True, dtype=dtype, **pre)
    a = to(cpu, DEV)
    bits = not (T == 5000 and dtype == torch.bfloat16 and columns % 2 == 1)
    views = {n: inside(a[n], 3 + i, 2, columns) for i, n in enumerate(("x", "g", "beta")) if n in a}
    want = kda.glr_fwd(**a)
    got = kda.glr_fwd(**(a | views))
    if bits:
        same(got, want)
    else:
        check_forward(cpu, *got, *glr_recurrent(**cpu))
    d_y = torch.randn_like(want[0])
    rest = {n: t for n, t in a.items() if n not in ("x", "g", "beta")}
    grads = [kda.glr_bwd(b["x"], b["g"], want[0], d_y, b.get("beta"), **rest) for b in (a, views)]
    if bits:
        same(*grads)
    else:
        y, d = want[0].cpu(), d_y.cpu()
        check_gradients(cpu, y, d, None, grads[1], glr_gradients(**cpu, y=y, d_y=d))
    rest.pop("initial_state")
    states = [a["initial_state"].clone() for _ in range(2)]
    same(*[(kda.glr_step(b["x"], b["g"], s, b.get("beta"), **rest),) for b, s in zip((a, views), states)])
    same(*[(s,) for s in states])


def test_the_last_tokens_of_a_long_buffer():
    """What a serving loop holds: one token a row, 2^23 elements apart, in a step, a forward and a differentiable call."""
    B, T, D = 3, 4096, 2048
    x, g = (torch.randn(B, T, D, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    g = -g.abs()
    state = torch.randn(B, D, device=DEV)
    keep = [state.clone() for _ in range(4)]
    last = lambda t: t[:, -1:]
    copy = lambda t: t[:, -1:].clone()
    assert torch.equal(kda.glr_step(last(x), last(g), keep[0]), kda.glr_step(copy(x), copy(g), keep[1]))
    assert torch.equal(keep[0], keep[1])
    for call in (kda.glr_fwd, kda.chunk_glr):
        same(call(last(x), last(g), initial_state=state), call(copy(x), copy(g), initial_state=state))
    leaf = x.clone().requires_grad_()
    y, _ = kda.chunk_glr(leaf[:, 100:300], g[:, 50:250])
    y.float().square().sum().backward()
    (dx,) = torch.autograd.grad(kda.chunk_glr(part := x[:, 100:300].clone().requires_grad_(), g[:, 50:250].clone())[0]
                                .float().square().sum(), [part])
    assert torch.equal(leaf.grad[:, 100:300], dx) and not leaf.grad[:, :100].any() and not leaf.grad[:, 300:].any()


def test_batches_that_overlap_or_interleave_are_refused():
    wide = torch.zeros(4, 6, 8, device=DEV)
    good = torch.zeros(2, 3, 8, device=DEV)
    for bad in (wide[:2, :3].transpose(0, 1).contiguous().transpose(0, 1)[:, :, :8], wide[:1, :3].expand(2, 3, 8),
                torch.as_strided(wide, (2, 3, 8), (16, 8, 1)), torch.as_strided(wide, (2, 3, 8), (48, 4, 1))):
        for call in (lambda: kda.glr_fwd(bad, good), lambda: kda.glr_step(good, bad, torch.zeros(2, 8, device=DEV))):
            with pytest.raises(ValueError, match="evenly spaced and rows of the batch one behind another"):
                call()
