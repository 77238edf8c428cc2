"""The words in which tiles of the gated linear recurrence hand over what they do to a state, on the CPU: the functions of
csrc/glr_tiles.h compiled for the host."""
from __future__ import annotations

import ctypes
import os
import subprocess

import numpy as np
import pytest

from chunked_kimi_delta_amd import build

SOURCE = """
#include "glr_tiles.h"
extern "C" void words(const float *c, const float *s, const float *E, int64_t n, uint64_t *w, float *c2, float *s2, float *E2)
{
    for (int64_t i = 0; i < n; ++i) {
        w[i] = glr::word_of(c[i], s[i], E[i]);
        glr::from_word(w[i], c2[i], s2[i], E2[i]);
    }
}
extern "C" void given_up(uint64_t w, uint64_t *as, float *c, float *s, float *E)
{
    *as = glr::met(w);
    glr::from_word(*as, *c, *s, *E);
}
"""


@pytest.fixture(scope="module")
def words(tmp_path_factory):
    d = tmp_path_factory.mktemp("words")
    src, out = d / "words.hip", d / "words.so"
    src.write_text(SOURCE)
    subprocess.run([build.hipcc(), *build.HIPCC_FLAGS, "-I", build.CSRC, "-shared", str(src), "-o", str(out)], check=True,
                   capture_output=True)
    lib = ctypes.CDLL(os.fspath(out))

    def call(c, s, E):
        c, s, E = (np.ascontiguousarray(np.broadcast_to(np.asarray(x, np.float32), np.shape(c))) for x in (c, s, E))
        w = np.zeros(len(c), np.uint64)
        back = [np.zeros(len(c), np.float32) for _ in range(3)]
        ptr = lambda a: a.ctypes.data_as(ctypes.c_void_p)
        lib.words(ptr(c), ptr(s), ptr(E), ctypes.c_int64(len(c)), ptr(w), *map(ptr, back))
        return (w, *back)
    call.lib = lib
    return call


def test_maps_survive(words):
    """c is e^g (s zero), or e^g - 1 (s one): to half a step of 23 bits, without a bias; s and E exactly."""
    first = np.float32(0.4375).view(np.uint32)
    bits = (first + np.arange(4096, dtype=np.uint32)).view(np.float32)
    for s, c in ((0.0, bits), (1.0, -bits)):
        E = np.linspace(-3e38, 3e38, len(c)).astype(np.float32)
        w, c2, s2, E2 = words(c, s, E)
        assert (w >> np.uint64(63) == 1).all() and (s2 == s).all() and (E2 == E).all()
        step = 2.0 ** -25                                   # of 24 bits, at 0.4375
        off = (c2.astype(np.float64) - c) / step
        assert np.abs(off).max() <= 1.0 and abs(off.mean()) <= 1e-3
    for c, s in ((0.0, 0.0), (1.0, 0.0), (0.0, 1.0), (-0.0, 1.0), (-0.5, 1.0), (-2.0 ** -100, 1.0), (2.0 ** 126, 0.0),
                 (np.inf, 0.0)):
        _, c2, s2, _ = words([c], s, 0.0)
        assert c2[0] + s2[0] == c + s and (c2[0] == c or c == 0), (c, s)


def test_numbers_that_are_none(words):
    nans = np.array([0x7fc00000, 0x7fffffff, 0x7f800002, 0xffc00000, 0xffffffff, 0x7fc00001], np.uint32).view(np.float32)
    w, c, _, E = words(nans, 0.0, nans)
    assert (w >> np.uint64(63) == 1).all() and np.isnan(c).all() and np.isnan(E).all()
    _, c, _, E = words(np.array([0.5, 0.5], np.float32), 0.0, np.array([np.inf, -np.inf], np.float32))
    assert (E == [np.inf, -np.inf]).all() and (c == 0.5).all()


def test_a_slight_growth_does_not_become_a_decay(words):
    """e^g - 1 above zero, as the least positive log decays and windows of them give it: a decay rounded to 24 bits (half a
    step is 2^-24) and in the word to 23 (2^-23)."""
    c = np.array([1e-12, 1e-9, 1.4e-8, 3e-8, 1.1e-7, 1e-6], np.float32)
    _, c2, s2, _ = words(c, 1.0, 0.0)
    a = c2.astype(np.float64) + s2
    assert (a >= 1.0).all() and (np.abs(a - 1.0 - c) <= 2.0 ** -24 + 2.0 ** -23).all()


def test_a_wait_that_gives_up_is_loud(words):
    """What has not come stands for NaN, as a map and as a state; what has come stays as it is."""
    def given_up(w):
        u, f = ctypes.c_uint64(), [ctypes.c_float() for _ in range(3)]
        words.lib.given_up(ctypes.c_uint64(w), ctypes.byref(u), *map(ctypes.byref, f))
        return u.value, *(x.value for x in f)
    w, c, s, E = given_up(0)
    assert w >> 63 and np.isnan(c) and np.isnan(E) and not np.isfinite(np.float32(c) + np.float32(s))
    (there, *_) = words(np.array([0.5], np.float32), 0.0, 3.0)
    assert given_up(int(there[0])) == (int(there[0]), 0.5, 0.0, 3.0)
    state = 1 << 63 | int(np.float32(-2.5).view(np.uint32))
    assert given_up(state)[0] == state and given_up(state)[3] == -2.5
