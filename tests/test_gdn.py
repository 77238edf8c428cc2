"""The gated delta rule and the 8-bit rows on the CPU: the oracle's pins (against the KDA oracle
with the decay repeated, and finite differences), and every refusal of the C ABI and the binding
(no call here reaches a GPU)."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import chunked_kimi_delta_amd as kda
from chunked_kimi_delta_amd import _lib
from chunked_kimi_delta_amd._lib import GdnArgs
from gdn_cases import make
from oracle.backward import kda_backward_recurrent
from oracle.gdn import gdn_gradients, gdn_recurrent
from oracle.recurrent import kda_recurrent


def wide(a):
    """KDA's arguments: the decay repeated over the key dims."""
    K = a["q"].shape[3]
    g = a["g"].double()[..., None].expand(*a["g"].shape, K)
    f = lambda x: None if x is None else x.double().numpy()
    return (f(a["q"]), f(a["k"]), f(a["v"]), g.numpy(), f(a["beta"]), None,
            f(a.get("initial_state")), None if "cu_seqlens" not in a else a["cu_seqlens"].numpy())


@pytest.mark.parametrize("kw", [dict(B=2, T=9, H=1, G=2, h0=True), dict(lens=[4, 0, 7], H=2, h0=True)])
def test_oracle_is_kda_with_one_decay(kw):
    a = make(K=64, V=64, dtype=torch.float32, **kw)
    o, fin = gdn_recurrent(**a)
    ro, rfin = kda_recurrent(*wide(a))
    np.testing.assert_allclose(o.numpy(), ro, rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(fin.numpy(), rfin, rtol=1e-12, atol=1e-13)
    d_o, dht = torch.randn(o.shape).double(), torch.randn(fin.shape).double()
    names = ("q", "k", "v", "g", "beta", "initial_state")
    kw2 = {"cu_seqlens": a["cu_seqlens"]} if "cu_seqlens" in a else {}
    got = gdn_gradients({n: a[n] for n in names}, d_o, dht, **kw2)
    ref = dict(zip(names, kda_backward_recurrent(*wide(a), d_o.numpy(), dht.numpy())))
    ref["g"] = ref["g"].sum(-1)
    for n in names:
        np.testing.assert_allclose(got[n].numpy(), ref[n], rtol=1e-9, atol=1e-11, err_msg=n)


@pytest.mark.parametrize("gate", ["softplus", "bounded"])
def test_oracle_gradients_against_differences(gate):
    a = make(T=5, H=1, G=2, K=64, V=64, dtype=torch.float32, raw=True, gate=gate, h0=True)
    a = {n: x.double() if torch.is_tensor(x) else x for n, x in a.items()}
    names = ("q", "k", "v", "g", "beta", "initial_state", "A_log", "dt_bias")
    rest = {n: x for n, x in a.items() if n not in names}
    gen = torch.Generator().manual_seed(1)
    d_o = torch.randn(a["v"].shape, generator=gen).double()
    dht = torch.randn(a["initial_state"].shape, generator=gen).double()
    grads = gdn_gradients({n: a[n] for n in names}, d_o, dht, **rest)

    def loss(b):
        o, fin = gdn_recurrent(**b)
        return float((o * d_o).sum() + (fin * dht).sum())
    for n in names:
        step = torch.randn(a[n].shape, generator=gen).double()
        e = 1e-5
        diff = (loss(a | {n: a[n] + e * step}) - loss(a | {n: a[n] - e * step})) / (2 * e)
        # central differences err by e^2 times the third derivative
        assert abs(diff - float((grads[n] * step).sum())) <= 1e-6 * max(1.0, abs(diff)), n


# ---------------------------------------------------------------------------------- refusals

@pytest.fixture(scope="module")
def lib():
    return kda.load()


FAKE = 1 << 40          # never dereferenced: the calls below are refused before any launch


def args(**kw):
    a = GdnArgs()
    d = dict(B=1, T=100, N=1, H=2, HV=4, K=128, V=64, io=0, q=FAKE, k=FAKE, v=FAKE, g=FAKE,
             beta=FAKE, o=FAKE)
    d.update(kw)
    for n, x in d.items():
        setattr(a, n, x)
    return a


BAD = [
    (dict(K=96), _lib.KDA_ERR_UNSUPPORTED), (dict(V=32), _lib.KDA_ERR_UNSUPPORTED),
    (dict(io=2), _lib.KDA_ERR_UNSUPPORTED), (dict(H=1, HV=32769), _lib.KDA_ERR_UNSUPPORTED),
    (dict(HV=3), _lib.KDA_ERR_INVALID_ARG), (dict(H=0), _lib.KDA_ERR_INVALID_ARG),
    (dict(B=0), _lib.KDA_ERR_INVALID_ARG), (dict(N=2), _lib.KDA_ERR_INVALID_ARG),
    (dict(T=-1), _lib.KDA_ERR_INVALID_ARG), (dict(q=None), _lib.KDA_ERR_INVALID_ARG),
    (dict(beta=FAKE + 8), _lib.KDA_ERR_INVALID_ARG), (dict(o=None), _lib.KDA_ERR_INVALID_ARG),
    (dict(initial_state=FAKE + 4), _lib.KDA_ERR_INVALID_ARG),
    (dict(gate=3, A_log=FAKE), _lib.KDA_ERR_UNSUPPORTED), (dict(gate=1), _lib.KDA_ERR_INVALID_ARG),
    (dict(gate=2, A_log=FAKE, gate_lower_bound=0.0), _lib.KDA_ERR_INVALID_ARG),
    (dict(gate=1, A_log=FAKE, dt_bias=FAKE + 2), _lib.KDA_ERR_INVALID_ARG),
]


@pytest.mark.parametrize("kw,status", BAD)
def test_calls_refuse_bad_arguments(lib, kw, status):
    for T in (100, 4):              # the chunked form and the recurrence
        a = args(**({"T": T} | kw))
        assert lib.gdn_fwd(ctypes.byref(a), FAKE, 1 << 40, None) == status
        assert lib.gdn_step(ctypes.byref(a), FAKE, FAKE, 4, None) == status
    assert lib.gdn_fwd(None, FAKE, 1 << 40, None) == _lib.KDA_ERR_INVALID_ARG


def test_packed_arguments(lib):
    assert lib.gdn_fwd(ctypes.byref(args(B=2, N=2, cu_seqlens=FAKE)), FAKE, 1 << 40, None) == _lib.KDA_ERR_INVALID_ARG
    assert lib.gdn_fwd(ctypes.byref(args(N=0, cu_seqlens=FAKE)), FAKE, 1 << 40, None) == _lib.KDA_ERR_INVALID_ARG
    assert lib.gdn_step(ctypes.byref(args(cu_seqlens=FAKE)), FAKE, FAKE, 4, None) == _lib.KDA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,status", BAD)
def test_backward_refuses_bad_arguments(lib, kw, status):
    if "o" in kw:
        return                      # not read by the backward
    call = lambda a, d_o=FAKE, dA=FAKE, outs=(FAKE,) * 5, ws=FAKE, n=1 << 50: lib.gdn_bwd(
        ctypes.byref(a), d_o, FAKE, ws, n, *outs, FAKE, dA, None, None)
    assert call(args(**kw)) == status
    if kw == dict(K=96):            # and what the backward alone takes
        a, bad = args(), _lib.KDA_ERR_INVALID_ARG
        assert call(a, d_o=None) == call(a, outs=(FAKE, None, FAKE, FAKE, FAKE)) == bad
        assert call(args(gate=1, A_log=FAKE), dA=None) == call(args(gate=1, A_log=FAKE), dA=FAKE + 2) == bad
        for io in (0, 1):
            a = args(io=io)
            need = lib.gdn_bwd_workspace_bytes(ctypes.byref(a))
            assert need > 0
            assert call(a, ws=None) == call(a, n=need - 1) == call(a, ws=FAKE + 16) == _lib.KDA_ERR_WORKSPACE


@pytest.mark.parametrize("kw,status", BAD)
def test_backward_from_checkpoints_refuses_bad_arguments(lib, kw, status):
    if "o" in kw:
        return
    call = lambda a, scale=FAKE, d_o=FAKE, ws=FAKE, n=1 << 50: lib.gdn_bwd_packed(
        ctypes.byref(a), FAKE, scale, FAKE, d_o, FAKE, ws, n, *(FAKE,) * 5, FAKE, FAKE, None, None)
    assert call(args(**kw)) == status
    if kw == dict(K=96):
        bad = _lib.KDA_ERR_INVALID_ARG
        assert call(args(), scale=None) == call(args(), scale=FAKE + 2) == call(args(), d_o=None) == bad
        for io in (0, 1):
            a = args(io=io)
            need, plain = (f(ctypes.byref(a)) for f in (lib.gdn_bwd_packed_workspace_bytes, lib.gdn_bwd_workspace_bytes))
            assert need >= plain + 100 * (2 * 2 * 128 + 4 * 64) * (4 if io else 2)
            assert call(a, ws=None) == call(a, n=need - 1) == call(a, ws=FAKE + 16) == _lib.KDA_ERR_WORKSPACE


@pytest.mark.parametrize("kw", [
    dict(T=1 << 28), dict(N=1 << 22, cu_seqlens=FAKE), dict(N=1 << 16, H=32, HV=32, cu_seqlens=FAKE),
    dict(io=1, T=1 << 21, H=32, HV=32), dict(B=1 << 21, N=1 << 21, T=17, H=1, HV=1)])
def test_launches_that_do_not_fit_are_refused(lib, kw):
    a = args(**kw)
    bwd = lib.gdn_bwd(ctypes.byref(a), FAKE, FAKE, FAKE, 1 << 62, *(FAKE,) * 6, None, None, None)
    assert lib.gdn_fwd(ctypes.byref(a), FAKE, 1 << 62, None) == bwd == _lib.KDA_ERR_UNSUPPORTED
    assert lib.gdn_fwd_workspace_bytes(ctypes.byref(a)) == lib.gdn_bwd_workspace_bytes(ctypes.byref(a)) == 0


def test_workspace(lib):
    need = lambda **kw: lib.gdn_fwd_workspace_bytes(ctypes.byref(args(**kw)))
    assert need() > 0 and need(T=16) == 0 and need(K=96) == 0
    assert need(T=16, cu_seqlens=FAKE) > 0
    # few heads and long sequences: room for the segments' ends behind the chunks' records
    records = lambda T, HV, N=1: (T // 64 + N) * HV * 25 * 1024
    assert need() == records(100, 4) and need(T=4096, H=64, HV=256) == records(4096, 256)
    assert need(T=4096, H=2, HV=2) > records(4096, 2)
    n = need()
    call = lambda ws, size: lib.gdn_fwd(ctypes.byref(args()), ws, size, None)
    assert call(None, n) == call(FAKE, n - 1) == call(FAKE + 16, n) == _lib.KDA_ERR_WORKSPACE


def test_step_refuses_bad_pools(lib):
    a = args(B=3, N=3, T=1)
    step = lambda state, index, slots: lib.gdn_step(ctypes.byref(a), state, index, slots, None)
    assert step(None, FAKE, 4) == step(FAKE + 4, FAKE, 4) == _lib.KDA_ERR_INVALID_ARG
    assert step(FAKE, FAKE + 2, 4) == step(FAKE, None, 2) == step(FAKE, FAKE, -1) == _lib.KDA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), _lib.KDA_ERR_INVALID_ARG), (dict(D=12), _lib.KDA_ERR_INVALID_ARG),
    (dict(D=0), _lib.KDA_ERR_INVALID_ARG), (dict(D=520), _lib.KDA_ERR_UNSUPPORTED),
    (dict(io=7), _lib.KDA_ERR_UNSUPPORTED), (dict(rows=1 << 36), _lib.KDA_ERR_UNSUPPORTED),
    (dict(rows=1 << 30, D=8), _lib.KDA_ERR_UNSUPPORTED),
    (dict(x=None), _lib.KDA_ERR_INVALID_ARG), (dict(x=FAKE + 8), _lib.KDA_ERR_INVALID_ARG),
    (dict(data=FAKE + 4), _lib.KDA_ERR_INVALID_ARG), (dict(scale=None), _lib.KDA_ERR_INVALID_ARG),
])
def test_act8_refuses_bad_arguments(lib, kw, status):
    d = dict(x=FAKE, io=0, rows=5, D=64, data=FAKE, scale=FAKE) | kw
    assert lib.act8_pack(d["x"], d["io"], d["rows"], d["D"], d["data"], d["scale"], None) == status
    assert lib.act8_unpack(d["data"], d["scale"], d["io"], d["rows"], d["D"], d["x"], None) == status


def test_binding_refuses_before_any_call():
    a = make(T=20, K=64, V=64)
    with pytest.raises(ValueError, match="HIP device"):
        kda.gdn_bwd(**a, d_o=a["v"])
    for fn in (kda.chunk_gdn, kda.chunk_kda):
        with pytest.raises(ValueError, match="HIP device"):
            fn(**a)
    with pytest.raises(ValueError, match="HIP device"):
        kda.gdn_fwd(**a)
    with pytest.raises(TypeError, match="io dtype"):
        kda.gdn_fwd(**{n: x.half() for n, x in a.items()})
    with pytest.raises(ValueError, match="HIP device"):
        kda.gdn_step(**a, state=torch.zeros(1, 1, 64, 64))
    with pytest.raises(ValueError, match="HIP device"):
        kda.pack8(torch.zeros(4, 64))
    with pytest.raises(TypeError, match="dtype"):
        kda.pack8(torch.zeros(4, 64, dtype=torch.float16))
    p = kda.Packed8(torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4), torch.bfloat16)
    with pytest.raises(ValueError, match="HIP device"):
        kda.unpack8(p)
    with pytest.raises(ValueError, match="one scale"):
        kda.unpack8(p._replace(scale=torch.zeros(3)))
    with pytest.raises(TypeError, match="int8"):
        kda.unpack8(p._replace(data=torch.zeros(4, 64)))
    p = {n: kda.Packed8(a[n].to(torch.int8), a[n][..., 0].float(), torch.bfloat16) for n in ("q", "k", "v")}
    with pytest.raises(ValueError, match="HIP device"):
        kda.gdn_bwd(**(a | p), d_o=a["v"])
    with pytest.raises(TypeError, match="all be checkpoints"):
        kda.GdnBwdPlan(**(a | {"q": p["q"]}), d_o=a["v"])
    with pytest.raises(TypeError, match="one dtype"):
        kda.gdn_bwd(**(a | p | {"k": p["k"]._replace(dtype=torch.float32)}), d_o=a["v"])
