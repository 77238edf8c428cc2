"""The README's example of a recurrence and of pools of states runs as it stands, and leaves every row in flight with the
slot of its own states."""
from __future__ import annotations

import os
import re

import pytest
import torch

import chunked_kimi_delta_amd as kda

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def test_example():
    code = [b for b in re.findall(r"```python\n(.*?)```", open(README).read(), re.S) if "pool_fork" in b][0]
    code = code[code.index("# one state a channel"):]
    B, T, D, HV, K = 5, 30, 64, 2, 64
    torch.manual_seed(1)
    n = lambda *s: torch.randn(*s, device=DEV)
    pools = [torch.zeros(9, HV, K, K, device=DEV), torch.zeros(9, D, device=DEV)]
    env = dict(torch=torch, kda=kda, x=n(B, T, D), g=n(B, T, D), beta=n(B, T, D), A_log=n(D), states=n(B, HV, K, K),
               gdn_pool=pools[0], glr_pool=pools[1], used=torch.zeros(9, dtype=torch.bool, device=DEV),
               x1=n(B, 1, D), g1=-n(B, 1, D).abs())
    env["used"][2] = True                                   # somebody else's
    pools[1][2] = 7.0
    env["x"].requires_grad_()
    with torch.no_grad():
        exec(code, env)
    torch.cuda.synchronize()
    rows = env["rows"].tolist()
    assert len(set(rows)) == 4 and set(rows) < set(range(5)) and env["used"].tolist() == [True] * 5 + [False] * 4
    h = env["h"].clone()
    kda.glr_step(env["x1"], env["g1"], h)
    for i, at in enumerate(rows):                           # rows 0 and 1, and their copies
        assert torch.equal(pools[0][at], env["states"][i % 2]) and torch.equal(pools[1][at], h[i % 2])
    (other,) = set(range(5)) - set(rows)
    assert (pools[1][other] == 7.0).all()
