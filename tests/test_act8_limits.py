"""The 8-bit rows' largest calls (CPU: every call here is refused). A launch has less than 2^32 threads, rows of 8
values take four each, and the last block's count in full."""
from __future__ import annotations

import pytest

import chunked_kimi_delta_amd as kda
from chunked_kimi_delta_amd import _lib

FAKE = 1 << 40          # never dereferenced


@pytest.mark.parametrize("rows", [(1 << 30) - 63, (1 << 30) - 1])
def test_launches_that_do_not_fit_are_refused(rows):
    assert kda.load().act8_pack(FAKE, 0, rows, 8, FAKE, FAKE, None) == _lib.KDA_ERR_UNSUPPORTED
