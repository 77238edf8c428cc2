"""The gated linear recurrence on the GPU where the exponential of a log decay overflows."""
from __future__ import annotations

import math

import pytest
import torch

import chunked_kimi_delta_amd as kda
from glr_cases import to

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_growth_beyond_the_finite_numbers_is_an_infinity(dtype):
    """e^g is infinite from g = 88.73 on; one token, so that nothing follows the infinity."""
    g = torch.tensor([80.0, 88.5, 89.0, 90.0, 95.0, 100.0, 105.0, 110.0, 111.0, 120.0, 1000.0, math.inf])
    D = len(g)
    a = to(dict(x=torch.ones(1, 1, D).to(dtype), g=g.expand(1, 1, D).contiguous().to(dtype)), DEV)
    h0 = torch.ones(1, D, device=DEV)
    state = h0.clone()
    want = torch.exp(a["g"][0, 0, :2].double())
    # half a step of y; for bf16 also the exponent's rounded product with log2 e, 128 * 2^-24 of the result at most
    half = 2.0 ** -8 + 2.0 ** -16 if dtype == torch.bfloat16 else 2.0 ** -21
    for y in (kda.glr_fwd(**a, initial_state=h0)[0], kda.glr_step(**a, state=state)):
        assert (y[0, 0, 2:] == math.inf).all() and torch.isfinite(y[0, 0, :2]).all()
        assert ((y[0, 0, :2].double() - want).abs() <= half * want).all()
    assert (state[0, 2:] == math.inf).all()
