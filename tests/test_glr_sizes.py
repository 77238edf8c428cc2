"""Sizes beyond the C ABI's 32-bit counts are refused by the binding of the gated linear recurrence and of the pools, and
not cut (CPU: tensors without memory of their own)."""
from __future__ import annotations

import pytest
import torch

import chunked_kimi_delta_amd as kda

MANY = (1 << 32) + 5            # cut to 32 bits this is 5


def test_tokens_and_rows():
    long = torch.zeros(1, 1, 1).expand(1, MANY, 1)
    wide = torch.zeros(1, 1, 1).expand(MANY, 1, 1)
    for x in (long, wide):
        for call in (lambda: kda.glr_fwd(x, x), lambda: kda.chunk_glr(x, x), lambda: kda.GlrBwdPlan(None, x, x, x),
                     lambda: kda.glr_step(x, x, torch.zeros(4, 1))):
            with pytest.raises(ValueError, match=r"at most 2\^31 - 1"):
                call()


def test_slots():
    t = torch.zeros(1, 2, 1)
    with pytest.raises(ValueError, match=r"at most 2\^31 - 1"):
        kda.glr_step(t, t, torch.empty(MANY, 1, device="meta"))
    pool = torch.empty(MANY, 1, dtype=torch.int8, device="meta")
    used, i = torch.empty(MANY, dtype=torch.bool, device="meta"), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: kda.pool_copy(pool, i, i), lambda: kda.pool_fork(pool, used, i), lambda: kda.pool_free(pool, used, i),
                 lambda: kda.pool_compact(pool, used, i), lambda: kda.pool_alloc(used, 2), lambda: kda.pool_free((), used, i)):
        with pytest.raises(ValueError, match=r"at most 2\^31 - 1"):
            call()
