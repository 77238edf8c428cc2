"""Strides from row to row of a batch in the C ABI of the gated linear recurrence (CPU: no call here reaches a GPU)."""
from __future__ import annotations

import ctypes

import pytest

import chunked_kimi_delta_amd as kda
from chunked_kimi_delta_amd import _lib
from test_glr import BAD, FAKE, NOT, args, back

WS = _lib.KDA_ERR_WORKSPACE
LONG = dict(B=2, N=2, T=5000, D=64)         # tiles, which ask for a workspace


@pytest.mark.parametrize("name", ["x_batch", "g_batch", "beta_batch"])
def test_batch_strides(name):
    lib = kda.load()
    calls = (lambda a: lib.glr_fwd(ctypes.byref(a), None, 0, None), lambda a: back(lib, a, ws=None, size=0))
    step = lambda a: lib.glr_step(ctypes.byref(a), None, FAKE, 4, None)          # refused behind the strides, for its pool
    span = 4999 * 64 + 64
    for value, status in ((span, WS), (1 << 40, WS), (0, WS), (span - 1, BAD), (64, BAD), (-1, BAD), (-(1 << 40), BAD)):
        a = args(**LONG, **{name: value})
        assert [c(a) for c in calls] == [status] * 2, value
        assert step(a) == BAD
    one = args(**(LONG | dict(B=1, N=1)), **{name: -1})                          # one row: not read
    assert [c(one) for c in calls] == [WS] * 2
    a = args(B=2, N=2, T=1, **{name: 63})
    assert lib.glr_fwd(ctypes.byref(a), None, 0, None) == lib.glr_step(ctypes.byref(a), FAKE, FAKE, 4, None) == BAD


def test_strides_from_token_to_token_have_their_limit_still():
    lib = kda.load()
    a = args(**LONG, **{"x_stride": (1 << 18) + 1, "x_batch": 1 << 31})
    assert lib.glr_fwd(ctypes.byref(a), None, 0, None) == NOT
