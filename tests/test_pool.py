"""Pools of states on the CPU: every refusal of the C ABI and the binding (no call here reaches a GPU)."""
from __future__ import annotations

import ctypes

import pytest
import torch

import chunked_kimi_delta_amd as kda
from chunked_kimi_delta_amd import _lib
from chunked_kimi_delta_amd._lib import PoolRef

FAKE = 1 << 40          # never dereferenced
OK, BAD, NOT, WS = _lib.KDA_OK, _lib.KDA_ERR_INVALID_ARG, _lib.KDA_ERR_UNSUPPORTED, _lib.KDA_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    return kda.load()


def refs(*pools):
    return (PoolRef * max(1, len(pools)))(*pools)


GOOD = (FAKE, 64)


def calls(lib, pools=(GOOD,), n_pools=None, slots=8, sources=None, m=0, used=FAKE, src=FAKE, dst=FAKE, n=4, count=FAKE,
          ws=FAKE, size=1 << 30):
    r = refs(*pools)
    np = len(pools) if n_pools is None else n_pools
    s = None if sources is None else (ctypes.c_void_p * len(sources))(*sources)
    return {
        "copy": lambda: lib.pool_copy(r, np, slots, s, m, src, dst, n, None),
        "fork": lambda: lib.pool_fork(r, np, slots, s, m, used, src, dst, n, None),
        "free": lambda: lib.pool_free(r, np, slots, used, src, n, None),
        "compact": lambda: lib.pool_compact(r, np, slots, used, src, n, count, ws, size, None),
    }


@pytest.mark.parametrize("kw,status", [
    (dict(n_pools=-1), BAD), (dict(slots=-1), BAD), (dict(n=-1), BAD), (dict(slots=(1 << 24) + 1), NOT),
    (dict(n=(1 << 24) + 1), NOT), (dict(pools=((None, 64),)), BAD), (dict(pools=((FAKE, 0),)), BAD),
    (dict(pools=(GOOD, (FAKE, -4))), BAD), (dict(pools=((FAKE, (1 << 39) + 1),)), NOT), (dict(src=FAKE + 2), BAD)])
def test_calls_refuse_bad_arguments(lib, kw, status):
    for name, call in calls(lib, **kw).items():
        assert call() == status, name


def test_calls_refuse_their_own(lib):
    for kw in (dict(dst=FAKE + 1), dict(sources=[None], m=3), dict(sources=[FAKE], m=-1)):
        for name in ("copy", "fork"):
            assert calls(lib, **kw)[name]() == BAD, (name, kw)
    assert calls(lib, sources=[FAKE], m=(1 << 24) + 1)["copy"]() == NOT
    assert calls(lib, dst=None)["fork"]() == BAD
    for name in ("fork", "free", "compact"):
        assert calls(lib, used=None)[name]() == BAD, name
    for name in ("free", "compact"):
        assert calls(lib, src=None)[name]() == BAD, name
    for kw in (dict(count=None), dict(count=FAKE + 2)):
        assert calls(lib, **kw)["compact"]() == BAD
    need = lib.pool_compact_workspace_bytes(8)
    assert need > 0 and lib.pool_compact_workspace_bytes(-1) == lib.pool_compact_workspace_bytes((1 << 24) + 1) == 0
    for kw in (dict(ws=None), dict(ws=FAKE + 128), dict(size=need - 1)):
        assert calls(lib, **kw)["compact"]() == WS
    assert lib.pool_copy(None, 1, 8, None, 0, FAKE, FAKE, 4, None) == BAD


def test_nothing_to_do(lib):
    for name in ("copy", "fork", "free"):
        assert calls(lib, n=0)[name]() == OK, name


def test_binding_refuses_before_any_call():
    p, used, i = torch.zeros(8, 4), torch.zeros(8, dtype=torch.bool), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: kda.pool_copy(p, i, i), lambda: kda.pool_fork(p, used, i), lambda: kda.pool_free(p, used, i),
                 lambda: kda.pool_compact(p, used, i), lambda: kda.pool_alloc(used, 2), lambda: kda.pool_free((), used, i)):
        with pytest.raises(ValueError, match="HIP device"):
            call()
    with pytest.raises(ValueError, match="contiguous"):
        kda.pool_copy(torch.zeros(4, 8).t(), i, i)
    with pytest.raises(ValueError, match="at least one pool"):
        kda.pool_copy((), i, i)
