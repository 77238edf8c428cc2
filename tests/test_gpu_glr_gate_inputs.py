"""Gate inputs of plus and minus infinity (a state cleared or kept) in the gated linear recurrence on the GPU."""
from __future__ import annotations

import math

import pytest
import torch

import chunked_kimi_delta_amd as kda
from glr_cases import make, to

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
LOWEST = {t: torch.finfo(t).min for t in (torch.bfloat16, torch.float32)}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [300, 5000])                  # strips and tiles
@pytest.mark.parametrize("gate", ["softplus", "bounded"])
@pytest.mark.parametrize("beta", [False, True])
def test_infinite_and_lowest_inputs_are_what_far_ones_are(beta, gate, T, dtype):
    """At 10^4 both gates have reached their ends, and their slopes are zero: an infinity, or the type's largest and
    lowest values, give the same bits in every output, the sums for A_log and dt_bias among them."""
    a = make(T=T, D=20, h0=True, sigmoid=beta, gate=gate, dtype=dtype)
    gen = torch.Generator().manual_seed(2)
    up, down = torch.rand(a["g"].shape, generator=gen) < 0.05, torch.rand(a["g"].shape, generator=gen) < 0.05
    up[0, 0, :3], down[0, -1, :3] = True, True
    d_y = torch.randn(a["g"].shape, generator=gen).to(dtype).to(DEV)
    outs = []
    for far in (1e4, math.inf, -LOWEST[dtype]):
        b = to(a | {"g": torch.where(down, -far, torch.where(up, far, a["g"].double())).to(dtype)}, DEV)
        y, fin = kda.glr_fwd(**b)
        outs.append((y, fin, *kda.glr_bwd(b.pop("x"), b.pop("g"), y, d_y, **b)))
    torch.cuda.synchronize()
    names = ("y", "final", "dx", "dg", "dbeta", "dh0", "dA_log", "ddt_bias")
    for other in outs[1:]:
        for n, p, q in zip(names, outs[0], other):
            assert p is None or (torch.isfinite(q).all() and torch.equal(p, q)), n
