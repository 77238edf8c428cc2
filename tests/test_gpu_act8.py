"""Rows kept in 8 bits on the GPU: the whole numbers, scales and values against their definition
in 64 bits, exactly (the rounding is decided exactly for bf16; fp32 rows are compared where the
quotient is further from a tie than a 64-bit division errs, which is everywhere here)."""
from __future__ import annotations

import pytest
import torch

import chunked_kimi_delta_amd as kda

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def define(x):
    y = x.double()
    m = y.abs().amax(-1, keepdim=True)
    n = torch.where(m > 0, torch.round(y * 127 / torch.where(m > 0, m, 1.0)), 0.0)
    return n.to(torch.int8), (m.squeeze(-1).float() / 127)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(1, 8), (5, 3, 64), (1000, 128), (7, 24), (3, 104), (2, 200), (9, 512), (0, 64)])
def test_round_trip(shape, dtype):
    gen = torch.Generator().manual_seed(shape[-1])
    x = (torch.randn(*shape, generator=gen) * torch.exp(2 * torch.randn(*shape[:-1], 1, generator=gen))).to(dtype)
    p = kda.pack8(x.to(DEV))
    y = kda.unpack8(p)
    torch.cuda.synchronize()
    if x.numel() == 0:
        assert y.shape == x.shape
        return
    n, s = define(x)
    assert torch.equal(p.data.cpu(), n) and torch.equal(p.scale.cpu(), s)
    assert y.dtype == dtype and torch.equal(y.cpu(), (n.float() * s[..., None]).to(dtype))
    # half a step of the row, then the io type's own rounding
    half = x.double().abs().amax(-1, keepdim=True) / 254
    tol = half * (1 + 1e-6) + torch.finfo(dtype).eps / 2 * x.double().abs() * 1.01 + half * 0.01
    assert ((y.cpu().double() - x.double()).abs() <= tol).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_ties_extremes_and_zero_rows(dtype):
    x = torch.zeros(7, 64, dtype=dtype)
    x[0, :4] = torch.tensor([127.0, 0.5, 1.5, -2.5])          # ties go to even
    x[1, 3] = torch.finfo(dtype).max                           # 127 x would overflow
    x[1, 4] = -torch.finfo(dtype).max / 2
    x[2, 5] = torch.finfo(dtype).tiny
    x[4, 0], x[4, 1] = 3.0, 1e-30
    x[5] = -1.0
    p = kda.pack8(x.to(DEV))
    n, s = define(x)
    assert torch.equal(p.data.cpu(), n) and torch.equal(p.scale.cpu(), s)
    assert p.data[0, 1:4].tolist() == [0, 2, -2]
    assert (kda.unpack8(p)[3] == 0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_bad_value_marks_its_row_only(bad):
    x = torch.randn(6, 64).bfloat16()
    clean = kda.unpack8(kda.pack8(x.to(DEV))).cpu()
    x[2, 7] = bad
    y = kda.unpack8(kda.pack8(x.to(DEV))).cpu()
    assert torch.isnan(y[2].float()).all()
    assert torch.equal(y[[0, 1, 3, 4, 5]], clean[[0, 1, 3, 4, 5]])


def test_replays_of_a_graph():
    x = torch.randn(100, 64, device=DEV).bfloat16()
    kda.unpack8(kda.pack8(x))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = kda.unpack8(kda.pack8(x))
    for seed in range(3):
        torch.manual_seed(seed)
        x.copy_(torch.randn(100, 64))
        want = kda.unpack8(kda.pack8(x))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_offsets_beyond_32_bits():
    rows, D = (1 << 25) + 5, 128                # 4.3e9 values: the last rows against a call of their own
    x = torch.empty(rows, D, dtype=torch.bfloat16, device=DEV).normal_()
    p = kda.pack8(x)
    tail = kda.pack8(x[-1000:].clone())
    assert torch.equal(p.data[-1000:], tail.data) and torch.equal(p.scale[-1000:], tail.scale)
    assert torch.equal(kda.unpack8(p)[-1000:], kda.unpack8(tail))


def test_other_streams():
    x = torch.randn(3000, 64, device=DEV).bfloat16()
    want = kda.unpack8(kda.pack8(x))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = kda.unpack8(kda.pack8(x))
    side.synchronize()
    assert torch.equal(y, want)
