"""Log decays above zero in the gated linear recurrence on the GPU, with sums far from overflow: within the bounds of the
recurrence (e^g is rounded to 24 bits, which one of their units counts)."""
from __future__ import annotations

import pytest
import torch

import chunked_kimi_delta_amd as kda
from glr_cases import check_forward, check_gradients, make, to
from oracle.glr import glr_gradients, glr_recurrent

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [1500, 5000])                 # strips and tiles
def test_states_that_grow_and_shrink(T, dtype):
    """In turn up and down by e^g a token, sums between 0 and 64, an own period and size a channel."""
    D = 12
    a = make(T=T, D=D, h0=True, dtype=dtype)
    period = torch.tensor([1, 2, 7, 16, 50, 64, 100, 128, 300, 512, 640, 800])
    size = torch.minimum(64.0 / period, torch.tensor(20.0))
    at = torch.arange(T)[:, None] // period
    a["g"] = torch.where(at % 2 == 0, size, -size)[None].to(dtype)
    y, fin = kda.glr_fwd(**to(a, DEV))
    check_forward(a, y, fin, *glr_recurrent(**a))
    gen = torch.Generator().manual_seed(3)
    d_y, dht = torch.randn(y.shape, generator=gen).to(dtype), torch.randn(fin.shape, generator=gen)
    b = to(a, DEV)
    got = kda.glr_bwd(b.pop("x"), b.pop("g"), y, d_y.to(DEV), dht=dht.to(DEV), **b)
    torch.cuda.synchronize()
    check_gradients(a, y.cpu(), d_y, dht, got, glr_gradients(**a, y=y.cpu(), d_y=d_y, dht=dht))
