"""Every width of the strips of the gated linear recurrence (8, 16, 32 and 64 lanes a token) with every pre-stage, in
the forward and the gradients."""
from __future__ import annotations

import pytest
import torch

import chunked_kimi_delta_amd as kda
from glr_cases import check_forward, check_gradients, make, to
from oracle.glr import glr_gradients, glr_recurrent

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
PRE = [dict(), dict(beta=True), dict(sigmoid=True, gate="softplus"), dict(sigmoid=True, gate="bounded"),
       dict(gate="softplus"), dict(gate="bounded", dt_bias=False)]


def lanes(N, D):
    """The widest strips that leave every compute unit a workgroup, at least 8 lanes."""
    cus, n = torch.cuda.get_device_properties(0).multi_processor_count, 64
    while n > 8 and N * -(-D // n) < cus:
        n //= 2
    return n


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pre", PRE, ids=lambda p: "-".join(map(str, p.values())) or "plain")
@pytest.mark.parametrize("width", [8, 16, 32, 64])
def test_forward_and_gradients(width, pre, dtype):
    lens = [3, 70, 0, 9] * 19 + [150, 1, 300, 65]             # 80; steps of 512, 256, 128 and 64 tokens
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    least = -(-cus // len(lens))                              # strips a sequence that fill the device
    D = 20 if width == 8 else (least - 1) * width + 2
    assert lanes(len(lens), D) == width
    a = make(lens=lens, D=D, h0=True, tail=3, dtype=dtype, **pre)
    y, fin = kda.glr_fwd(**to(a, DEV))
    torch.cuda.synchronize()
    check_forward(a, y, fin, *glr_recurrent(**a))
    gen = torch.Generator().manual_seed(6)
    d_y, dht = torch.randn(y.shape, generator=gen).to(dtype), torch.randn(fin.shape, generator=gen)
    y[:, sum(lens):] = 0
    b = to(a, DEV)
    got = kda.glr_bwd(b.pop("x"), b.pop("g"), y, d_y.to(DEV), dht=dht.to(DEV), **b)
    torch.cuda.synchronize()
    y = y.cpu()
    check_gradients(a, y, d_y, dht, got, glr_gradients(**a, y=y, d_y=d_y, dht=dht))
