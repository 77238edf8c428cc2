"""The gated linear recurrence on the GPU: packed sequences that tiles take against the same sequences alone in strips,
and the bf16 gradients of the whole, forward and backward, against 64 bits."""
from __future__ import annotations

import pytest
import torch

import chunked_kimi_delta_amd as kda
from glr_cases import STEPS, _active, _scan_bound, check, forward_bound, make, to
from oracle.glr import glr_gradients, glr_recurrent

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def decay_bound(a, d_y, ref, exact):
    """Bounds of dg's errors (before its rounding) for one bf16 sequence without a gate, from the errors of m and of the
    states: the backward reads the forward's, which are its errors and half a step off the exact ones."""
    g, _ = _active(a)
    D = g.shape[2]
    e, dy = torch.exp(g).reshape(-1, D), d_y.double().reshape(-1, D)
    unit = STEPS[a["g"].dtype]
    bd, _, mag = _scan_bound(e, dy, torch.zeros(1, D, dtype=torch.float64), [(0, len(dy))], unit, reverse=True)
    m, bm = (e * ref["dh"].reshape(-1, D)).abs(), e * bd + unit * e * mag
    by, _ = forward_bound(a)
    states = exact[0].abs()
    before = torch.cat([a["initial_state"].double().abs(), states[:-1]])
    off = torch.cat([torch.zeros(1, D, dtype=torch.float64), (2.0 ** -8 * (states + by[0]) + by[0])[:-1]])
    return (off * (m + bm) + before * bm)[None]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_packed_sequences_are_what_they_are_alone(dtype):
    """Both err by their bounds, and bf16 outputs by half a step each."""
    lens = [1300] * 66
    lens[3], lens[4], lens[40] = 0, 2600, 1029
    a = make(lens=lens, D=3, h0=True, dtype=dtype)
    b = to(a, DEV)
    y, fin = kda.glr_fwd(**b)
    d_y = torch.randn_like(y)
    dx, dg, _, dh0, _, _ = kda.glr_bwd(b["x"], b["g"], y, d_y, cu_seqlens=b["cu_seqlens"], initial_state=b["initial_state"])
    bf16 = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    unit = STEPS[dtype]
    for s in (0, 3, 4, 40, 62, 63, 64, 65):
        lo, hi = int(a["cu_seqlens"][s]), int(a["cu_seqlens"][s + 1])
        if hi == lo:
            assert torch.equal(fin[s], b["initial_state"][s]) and (dh0[s] == 0).all()
            continue
        one = {n: b[n][:, lo:hi].contiguous() for n in ("x", "g")} | {"initial_state": b["initial_state"][s:s + 1]}
        y1, f1 = kda.glr_fwd(**one)
        x1, g1, _, h1, _, _ = kda.glr_bwd(None, one["g"], y[:, lo:hi].contiguous(), d_y[:, lo:hi].contiguous(),
                                          initial_state=one["initial_state"])
        cpu = to(one, "cpu")
        by, bf = forward_bound(cpu)
        d = lambda t: t.double().cpu()
        twice = lambda bound, t: 2 * bound + bf16 * (d(t).abs() + bound)
        check(y[:, lo:hi], d(y1), twice(by, y1), dtype, "y")
        check(fin[s:s + 1], d(f1), 2 * bf, torch.float32, "final")
        e = torch.exp(cpu["g"][0].double())
        bd, bend, mag = _scan_bound(e, d(d_y[0, lo:hi]), torch.zeros(1, 3, dtype=torch.float64), [(0, hi - lo)], unit, reverse=True)
        check(dx[:, lo:hi], d(x1), twice((bd + unit * mag)[None], x1), dtype, "dx")
        before = torch.cat([cpu["initial_state"].double(), d(y[0, lo:hi - 1])]).abs()
        check(dg[:, lo:hi], d(g1), twice((before * (e * bd + unit * e * mag))[None], g1), dtype, "dg")
        check(dh0[s:s + 1], d(h1), 2 * bend, torch.float32, "dh0")


@pytest.mark.parametrize("T", [200, 4096])
def test_gradients_of_bf16_through_the_forward(T):
    """dg takes the states from y as the forward rounded it: against the gradient in 64 bits, whose states are exact."""
    a = make(T=T, D=16, h0=True)
    b = to(a, DEV)
    y, _ = kda.glr_fwd(**b)
    d_y = torch.randn(y.shape, generator=torch.Generator().manual_seed(4)).bfloat16()
    dg = kda.glr_bwd(b.pop("x"), b.pop("g"), y, d_y.to(DEV), **b)[1]
    exact, _ = glr_recurrent(**a)
    ref = glr_gradients(**a, y=exact, d_y=d_y)
    check(dg, ref["g"], decay_bound(a, d_y, ref, exact), torch.bfloat16, "dg")
