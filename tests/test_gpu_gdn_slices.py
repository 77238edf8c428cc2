"""Calls on some tokens of a longer batch, whose g and beta need not begin at a multiple of 16 bytes: the results are
those of copies that do."""
from __future__ import annotations

import pytest
import torch

import chunked_kimi_delta_amd as kda
from gdn_cases import make, to

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SEQ = ("q", "k", "v", "g", "beta")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("i,j", [(1, 2), (3, 8), (5, 70)])
def test_tokens_of_a_longer_batch(i, j, dtype):
    a = to(make(T=80, H=1, G=2, K=64, V=64, dtype=dtype), DEV)
    part = {n: a[n][:, i:j] for n in SEQ}
    assert part["beta"].data_ptr() % 16 and part["beta"].is_contiguous()
    copy = {n: x.clone() for n, x in part.items()}
    state = [torch.full((1, 2, 64, 64), 0.1, device=DEV) for _ in range(2)]
    d_o = torch.randn_like(copy["v"])
    leaves = [{n: x.detach().requires_grad_() for n, x in d.items()} for d in (part, copy)]
    calls = (lambda d, s, _: (kda.gdn_step(**d, state=s), s), lambda d, s, _: kda.gdn_fwd(**d, initial_state=s),
             lambda d, s, _: kda.gdn_bwd(**d, d_o=d_o, initial_state=s)[:6],
             lambda d, s, x: torch.autograd.grad(kda.chunk_gdn(**x)[0], list(x.values()), d_o))
    for n, call in enumerate(calls):
        got, want = (call(d, s, x) for d, s, x in zip((part, copy), state, leaves))
        for x, y in zip(got, want):
            assert torch.equal(x, y), n


def test_a_plan_on_such_tokens_is_refused():
    a = to(make(T=80, H=1, G=2, K=64, V=64), DEV)
    with pytest.raises(RuntimeError, match="invalid argument"):
        kda.GdnFwdPlan(**{n: a[n][:, 1:70] for n in SEQ})()
