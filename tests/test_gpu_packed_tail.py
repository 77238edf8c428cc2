"""Rows behind the last packed sequence, in the differentiable calls: zero in o and in every gradient, whatever the
memory held before and whatever the inputs hold there."""
from __future__ import annotations

import pytest
import torch

import chunked_kimi_delta_amd as kda
from chunked_kimi_delta_amd.api import _zero_tail
from gdn_cases import make, to

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("checkpoint", [None, "int8"])
@pytest.mark.parametrize("G", [1, 2])
def test_chunk_kda_rows_behind_the_last_sequence_are_zero(G, checkpoint, dtype):
    a = to(make(lens=[70, 0, 100], H=2, G=G, K=64, V=64, tail=30, dtype=dtype), DEV)
    a["g"] = a["g"][..., None].expand(-1, -1, -1, 64).contiguous()
    names = ("q", "k", "v", "g", "beta")
    for n in names:
        a[n][:, 170:] = float("nan")            # read by nothing
    d_o = torch.randn_like(a["v"].float()).to(dtype)
    leaves = {n: a[n].clone().requires_grad_() for n in names}
    poison = [torch.full(a[n].shape, float("nan"), device=DEV, dtype=t) for n in names
              for t in (dtype, torch.float32) for _ in range(3)]
    del poison                                  # new tensors may well start as these
    o, _ = kda.chunk_kda(**leaves, cu_seqlens=a["cu_seqlens"], checkpoint=checkpoint)
    o.backward(d_o)
    assert (o[:, 170:] == 0).all() and torch.isfinite(o).all()
    cut = {n: a[n][:, :170].contiguous().requires_grad_() for n in names}
    want, _ = kda.chunk_kda(**cut, cu_seqlens=a["cu_seqlens"], checkpoint=checkpoint)
    want.backward(d_o[:, :170].contiguous())
    assert torch.equal(o[:, :170], want)
    for n, x in leaves.items():
        assert (x.grad[:, 170:] == 0).all() and torch.equal(x.grad[:, :170], cut[n].grad), n


@pytest.mark.parametrize("ends", [[0, 5, 9], [0, 0], [0, 3, 3, 40], [0, 1]])
@pytest.mark.parametrize("T", [0, 1, 9, 40])
def test_zero_tail_clears_the_rows_behind_and_nothing_else(T, ends):
    # rows of every size modulo a store, in one launch
    cu = torch.tensor([min(e, T) for e in ends], device=DEV)
    shapes = [(torch.bfloat16, (1,)), (torch.bfloat16, (3,)), (torch.float32, (1,)), (torch.float32, (5,)),
              (torch.bfloat16, (2, 64)), (torch.float32, (3, 128))]
    pads = [torch.full((1, T + 8, *s), 7.0, dtype=t, device=DEV) for t, s in shapes]
    views = [x[:, :T] for x in pads]                            # whatever follows the last row stays
    _zero_tail(cu, *views)
    torch.cuda.synchronize()
    at = int(cu[-1])
    for x in pads:
        assert (x[:, :at] == 7).all() and (x[:, at:T] == 0).all() and (x[:, T:] == 7).all()


def test_zero_tail_far_rows_streams_and_graphs():
    T, row = (1 << 20) + 3, 4096 + 2                            # beyond 2^32 bytes
    x = torch.full((1, T, row // 2), 1.0, dtype=torch.bfloat16, device=DEV)
    cu = torch.tensor([0, T - 2], device=DEV)
    _zero_tail(cu, x)
    assert (x[:, T - 2:] == 0).all() and (x[:, T - 1000:T - 2] == 1).all() and (x[:, :1000] == 1).all()
    y = torch.full((1, 10, 3), 1.0, device=DEV)
    cu = torch.tensor([0, 10], device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _zero_tail(cu, y)
    for end in (7, 2, 10):
        y.fill_(1.0)
        cu[1] = end
        graph.replay()
        torch.cuda.synchronize()
        assert (y[:, :end] == 1).all() and (y[:, end:] == 0).all()
