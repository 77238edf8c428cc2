"""Second derivatives through chunk_kda are refused: its backward is a kernel call that autograd sees nothing of, and
without the refusal they would come out as if the gradients were constants."""
from __future__ import annotations

import pytest
import torch

import chunked_kimi_delta_amd as kda
from gdn_cases import make, to

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("checkpoint", [None, "int8"])
def test_second_derivatives_are_refused(checkpoint):
    a = to(make(T=20, H=1, K=64, V=64, dtype=torch.float32), DEV)
    a["g"] = a["g"][..., None].expand(-1, -1, -1, 64).contiguous()
    q = a["q"].clone().requires_grad_()
    o, _ = kda.chunk_kda(**(a | {"q": q}), checkpoint=checkpoint)
    dq, = torch.autograd.grad(o.square().sum(), q, create_graph=True)
    plain, = torch.autograd.grad(kda.chunk_kda(**(a | {"q": q}), checkpoint=checkpoint)[0].square().sum(), q)
    assert torch.equal(dq, plain)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        dq.sum().backward()
