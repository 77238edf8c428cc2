"""gdn_zero_tail's refusals (CPU: no call here reaches a GPU)."""
from __future__ import annotations

import ctypes

import pytest

import chunked_kimi_delta_amd as kda
from chunked_kimi_delta_amd import _lib

FAKE = 1 << 40          # never dereferenced


@pytest.mark.parametrize("kw,status", [
    (dict(cu=None), _lib.KDA_ERR_INVALID_ARG), (dict(cu=FAKE + 4), _lib.KDA_ERR_INVALID_ARG),
    (dict(N=0), _lib.KDA_ERR_INVALID_ARG), (dict(T=-1), _lib.KDA_ERR_INVALID_ARG),
    (dict(x=[FAKE, None]), _lib.KDA_ERR_INVALID_ARG), (dict(x=[FAKE, FAKE + 4]), _lib.KDA_ERR_INVALID_ARG),
    (dict(rows=[2, 3]), _lib.KDA_ERR_INVALID_ARG), (dict(rows=[0, 2]), _lib.KDA_ERR_INVALID_ARG),
    (dict(rows=[2, 1 << 60]), _lib.KDA_ERR_INVALID_ARG),
    (dict(x=[FAKE] * 9, rows=[2] * 9), _lib.KDA_ERR_UNSUPPORTED),
    (dict(T=0), _lib.KDA_OK), (dict(x=[], rows=[]), _lib.KDA_OK),
])
def test_refusals(kw, status):
    d = dict(cu=FAKE, N=2, T=10, x=[FAKE, FAKE], rows=[2, 256]) | kw
    n = len(d["x"])
    assert kda.load().gdn_zero_tail(d["cu"], d["N"], d["T"], n, (ctypes.c_void_p * n)(*d["x"]),
                                    (ctypes.c_int64 * n)(*d["rows"]), None) == status


def test_missing_arrays():
    assert kda.load().gdn_zero_tail(FAKE, 1, 10, 1, None, None, None) == _lib.KDA_ERR_INVALID_ARG
