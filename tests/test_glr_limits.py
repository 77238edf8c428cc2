"""The launch limit that include/glr.h states for the gated linear recurrence: 2^23 workgroups and more are refused (CPU:
calls that are refused before any launch)."""
from __future__ import annotations

import ctypes

import pytest

import chunked_kimi_delta_amd as kda
from test_glr import FAKE, NOT, args, back


@pytest.mark.parametrize("kw", [
    dict(B=1 << 18, N=1 << 18, T=7, D=2048),                        # strips: N ceil(D / 64) = 2^23
    dict(T=100, D=2048, N=1 << 18, cu_seqlens=FAKE),
    dict(T=1 << 30, D=2048, cu_seqlens=FAKE),                       # tiles: (T / 64 + N) ceil(D / 64) > 2^23
])
def test_launches_of_two_to_the_23_workgroups(kw):
    lib = kda.load()
    a = args(**kw, x_stride=kw["D"], g_stride=kw["D"], beta_stride=kw["D"])
    assert lib.glr_fwd(ctypes.byref(a), FAKE, 1 << 62, None) == back(lib, a, size=1 << 62) == NOT
