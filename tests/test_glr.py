"""The gated linear recurrence on the CPU: the oracle's formulas (against autograd and differences) and every
refusal of the C ABI and the binding (no call here reaches a GPU)."""
from __future__ import annotations

import ctypes

import pytest
import torch

import chunked_kimi_delta_amd as kda
from chunked_kimi_delta_amd import _lib
from chunked_kimi_delta_amd._lib import GlrArgs
from glr_cases import make
from oracle.glr import glr_gradients, glr_recurrent

FAKE = 1 << 40          # never dereferenced: the calls below are refused before any launch
BAD, NOT = _lib.KDA_ERR_INVALID_ARG, _lib.KDA_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(B=2, T=7, D=3, h0=True), dict(lens=[3, 0, 4], D=2, h0=True, sigmoid=True),
                                dict(T=5, D=4, beta=True, gate="softplus"),
                                dict(T=5, D=4, sigmoid=True, gate="bounded", h0=True)])
def test_oracle_gradients(kw):
    a = make(dtype=torch.float32, **kw)
    a = {n: x.double() if torch.is_tensor(x) and x.is_floating_point() else x for n, x in a.items()}
    names = [n for n in ("x", "g", "beta", "initial_state", "A_log", "dt_bias") if n in a]
    leaves = {n: a[n].clone().requires_grad_() for n in names}
    y, fin = glr_recurrent(**(a | leaves))
    gen = torch.Generator().manual_seed(1)
    d_y, dht = (torch.randn(t.shape, generator=gen).double() for t in (y, fin))
    auto = dict(zip(names, torch.autograd.grad((y * d_y).sum() + (fin * dht).sum(), list(leaves.values()))))
    ref = glr_gradients(**a, y=y.detach(), d_y=d_y, dht=dht)
    for n in names:
        torch.testing.assert_close(ref[n], auto[n], rtol=1e-11, atol=1e-12)

    def loss(b):
        y, fin = glr_recurrent(**b)
        return float((y * d_y).sum() + (fin * dht).sum())
    for n in names:
        step = torch.randn(a[n].shape, generator=gen).double()
        e = 1e-5
        diff = (loss(a | {n: a[n] + e * step}) - loss(a | {n: a[n] - e * step})) / (2 * e)
        # central differences err by e^2 times the third derivative
        assert abs(diff - float((ref[n] * step).sum())) <= 1e-6 * max(1.0, abs(diff)), n


# ---------------------------------------------------------------------------------- refusals

@pytest.fixture(scope="module")
def lib():
    return kda.load()


def args(**kw):
    a = GlrArgs()
    d = dict(B=1, T=100, N=1, D=64, io=0, x=FAKE, g=FAKE, beta=FAKE, y=FAKE, x_stride=64, g_stride=64, beta_stride=64)
    d.update(kw)
    for n, x in d.items():
        setattr(a, n, x)
    return a


SHARED = [
    (dict(D=0), BAD), (dict(B=0), BAD), (dict(T=-1), BAD), (dict(N=2), BAD), (dict(io=2), NOT),
    (dict(D=(1 << 18) + 1, x_stride=1 << 19, g_stride=1 << 19, beta_stride=1 << 19), NOT),
    (dict(g_stride=(1 << 18) + 1), NOT), (dict(beta_stride=(1 << 18) + 1), NOT),
    (dict(g=None), BAD), (dict(y=None), BAD), (dict(x=None), BAD), (dict(x_stride=63), BAD), (dict(g_stride=0), BAD),
    (dict(beta_stride=-64), BAD), (dict(g=FAKE + 1), BAD), (dict(beta=FAKE + 1), BAD), (dict(io=1, x=FAKE + 2), BAD),
    (dict(gate=3, A_log=FAKE), NOT), (dict(gate=1), BAD), (dict(gate=1, A_log=FAKE + 2), BAD),
    (dict(gate=1, A_log=FAKE, dt_bias=FAKE + 2), BAD), (dict(gate=2, A_log=FAKE, gate_lower_bound=0.0), BAD),
    (dict(gate=2, A_log=FAKE, gate_lower_bound=float("-inf")), BAD),
    (dict(gate=2, A_log=FAKE, gate_lower_bound=float("nan")), BAD),
]


def back(lib, a, d_y=FAKE, dht=None, ws=FAKE, size=1 << 50, dx=FAKE, dg=FAKE, dbeta=FAKE, dh0=None, dA=FAKE, db=None):
    return lib.glr_bwd(ctypes.byref(a), d_y, dht, ws, size, dx, dg, dbeta, dh0, dA, db, None)


@pytest.mark.parametrize("kw,status", SHARED)
def test_calls_refuse_bad_arguments(lib, kw, status):
    a = args(**kw)
    assert lib.glr_fwd(ctypes.byref(a), FAKE, 1 << 50, None) == status
    assert lib.glr_step(ctypes.byref(a), FAKE, FAKE, 4, None) == status
    assert back(lib, a) == status


def test_null_arguments(lib):
    assert lib.glr_fwd(None, None, 0, None) == lib.glr_step(None, FAKE, FAKE, 4, None) == BAD
    assert lib.glr_bwd(None, *(FAKE,) * 3, 0, *(FAKE,) * 6, None) == BAD
    assert lib.glr_fwd_workspace_bytes(None) == lib.glr_bwd_workspace_bytes(None) == 0


def test_packed_arguments(lib):
    for kw in (dict(B=2, N=2), dict(N=0), dict(cu_seqlens=FAKE + 4)):
        a = args(**(dict(cu_seqlens=FAKE) | kw))
        assert lib.glr_fwd(ctypes.byref(a), FAKE, 1 << 50, None) == back(lib, a) == BAD
    assert lib.glr_step(ctypes.byref(args(cu_seqlens=FAKE)), FAKE, FAKE, 4, None) == BAD


def test_launches_that_do_not_fit_are_refused(lib):
    a = args(D=4096, x_stride=4096, g_stride=4096, beta_stride=4096, N=1 << 20, cu_seqlens=FAKE)
    assert lib.glr_fwd(ctypes.byref(a), FAKE, 1 << 50, None) == back(lib, a) == NOT
    a = args(T=1 << 30, D=1 << 12, x_stride=4096, g_stride=4096, beta_stride=4096)      # tiles
    assert lib.glr_fwd(ctypes.byref(a), FAKE, 1 << 60, None) == back(lib, a, size=1 << 60) == NOT
    a = args(B=1 << 30, N=1 << 30, T=1)
    assert lib.glr_step(ctypes.byref(a), FAKE, FAKE, 1, None) == NOT


def test_backward_refuses_bad_arguments(lib):
    a = args()
    for kw in (dict(d_y=None), dict(dx=None), dict(dg=None), dict(dbeta=None), dict(d_y=FAKE + 1), dict(dx=FAKE + 1),
               dict(dht=FAKE + 2), dict(dh0=FAKE + 2)):
        assert back(lib, a, **kw) == BAD, kw
    g = args(gate=1, A_log=FAKE)
    assert back(lib, g, dA=None) == back(lib, g, dA=FAKE + 2) == back(lib, g, db=FAKE + 2) == BAD
    need = lib.glr_bwd_workspace_bytes(ctypes.byref(g))
    assert need > 0
    for kw in (dict(ws=None), dict(size=need - 1), dict(ws=FAKE + 64)):
        assert back(lib, g, **kw) == _lib.KDA_ERR_WORKSPACE, kw


def test_workspace(lib):
    long = dict(D=2048, x_stride=2048, g_stride=2048, beta_stride=2048)
    fwd = lambda **kw: lib.glr_fwd_workspace_bytes(ctypes.byref(args(**kw)))
    bwd = lambda **kw: lib.glr_bwd_workspace_bytes(ctypes.byref(args(**kw)))
    assert fwd() == bwd() == fwd(D=0) == bwd(D=0) == 0          # strips, and refused
    assert bwd(gate=1) >= 2 * 64 * 4                            # partial sums of the gate's gradients
    # tiles of 64 tokens (with beta), a word of 8 bytes a channel each
    assert fwd(T=1 << 16, **long) >= (1 << 10) * 2048 * 8 and bwd(T=1 << 16, **long) >= (1 << 10) * 2048 * 8
    assert fwd(T=1 << 16, beta=None, **long) >= (1 << 9) * 2048 * 8
    a = args(T=1 << 16, **long)
    for call, need in ((lambda ws, n: lib.glr_fwd(ctypes.byref(a), ws, n, None), fwd(T=1 << 16, **long)),
                       (lambda ws, n: back(lib, a, ws=ws, size=n), bwd(T=1 << 16, **long))):
        assert call(None, need) == call(FAKE, need - 1) == call(FAKE + 64, need) == _lib.KDA_ERR_WORKSPACE


def test_step_refuses_bad_pools(lib):
    a = args(B=3, N=3, T=1)
    step = lambda state, index, slots: lib.glr_step(ctypes.byref(a), state, index, slots, None)
    assert step(None, FAKE, 4) == step(FAKE + 2, FAKE, 4) == BAD
    assert step(FAKE, FAKE + 2, 4) == step(FAKE, None, 2) == step(FAKE, FAKE, -1) == BAD


def test_calls_of_no_tokens_or_sequences_are_fine(lib):
    a = args(T=0, x=None, g=None, y=None)
    assert lib.glr_step(ctypes.byref(a), FAKE, FAKE, 4, None) == 0


def test_binding_refuses_before_any_call():
    a = make(T=20, D=8, beta=True)
    b = dict(y=a["x"], d_y=a["x"])
    for fn, kw in ((kda.glr_fwd, {}), (kda.chunk_glr, {}), (kda.glr_bwd, b),
                   (kda.glr_step, dict(state=torch.zeros(1, 8)))):
        with pytest.raises(ValueError, match="HIP device"):
            fn(**a, **kw)
        with pytest.raises(TypeError, match="io dtype"):
            fn(**{n: x.half() for n, x in a.items()}, **kw)
    with pytest.raises(ValueError, match="x is needed"):
        kda.glr_bwd(None, a["g"], beta=a["beta"], **b)
