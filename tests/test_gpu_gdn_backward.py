"""Gradients of the gated delta rule on the GPU against autograd through the fp64 token recurrence
(oracle/gdn.py), the autograd functions and their 8-bit checkpoints.

Bars, relative L2 of each gradient. bf16 io: a path from the inputs to a gradient has at most four
values rounded to bf16 (S or dS', e or dR, a 64 x 64 matrix, the gradient itself); a rounding is off
by at most 2^-8 of the value, evenly spread, so by 2^-8 / sqrt(3) on the mean, and four by
2^-8 sqrt(4 / 3) = 4.5e-3: 2^-7. dg, dbeta (and the gate parameters') are differences of such sums
and may be a few times smaller than they: 2^-6. A single element has 2^-8 of itself, and of its row
(whose products it sums; rows may differ by orders of magnitude, so the tensor's rms alone would say
nothing of a large row) five times the mean of three roundings, 5 x 2^-8 rms: 2^-4 of the larger of
the row's and the tensor's rms. dh0 travels in two parts (17 bits): 2^-13. fp32 io: fp32 sums of up to 128 terms, ten behind
each other through both passes (2^-24 x 4.6 x sqrt(10) = 9e-7), that two inverses enlarge a few times
each: 2^-16."""
from __future__ import annotations

import pytest
import torch

import chunked_kimi_delta_amd as kda
from errlog import report_named
from gdn_cases import make, to
from oracle.gdn import gdn_gradients, gdn_recurrent

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, FP = torch.bfloat16, torch.float32
LEAVES = ("q", "k", "v", "g", "beta", "initial_state", "A_log", "dt_bias")
OUTS = ("q", "k", "v", "g", "beta", "initial_state", "A_log", "dt_bias")


def tol(name, dtype):
    if dtype == FP:
        return 2.0 ** -16
    return {"initial_state": 2.0 ** -13, "g": 2.0 ** -6, "beta": 2.0 ** -6, "A_log": 2.0 ** -6,
            "dt_bias": 2.0 ** -6}.get(name, 2.0 ** -7)


def cotangents(a, dht=True, seed=5):
    gen = torch.Generator().manual_seed(seed)
    d_o = torch.randn(a["v"].shape, generator=gen).to(a["v"].dtype)
    N = len(a["cu_seqlens"]) - 1 if "cu_seqlens" in a else a["q"].shape[0]
    shape = (N, a["v"].shape[2], a["q"].shape[3], a["v"].shape[3])
    return d_o, torch.randn(shape, generator=gen) if dht else None


def compare(got, ref, dtype, rows=None):
    errs = {}
    for n, want in ref.items():
        x = got[n].double().cpu()
        if rows is not None and n in ("q", "k", "v", "g", "beta"):
            x, want = x[:, :rows], want[:, :rows]
        assert x.shape == want.shape and torch.isfinite(x).all(), n
        size = want.norm()
        errs[n] = float((x - want).norm() / size.clamp_min(1e-30))
        if size == 0:
            assert (x == 0).all(), n
            continue
        assert errs[n] <= tol(n, dtype), f"{n}: {errs[n]:.3e}"
        rms = want.square().mean().sqrt()
        if n in ("q", "k", "v", "initial_state"):
            rms = torch.maximum(rms, want.square().mean(-1, keepdim=True).sqrt())
        assert ((x - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -4 * rms).all(), f"{n}: one element"
    report_named(**errs)


def check(a, dht=True, rows=None):
    d_o, dh = cotangents(a, dht)
    want0 = "initial_state" in a
    out = kda.gdn_bwd(**to(a, DEV), d_o=d_o.to(DEV), dht=None if dh is None else dh.to(DEV), want_dh0=want0)
    torch.cuda.synchronize()
    got = dict(zip(OUTS, out))
    leaves = {n: a[n] for n in LEAVES if a.get(n) is not None}
    rest = {n: x for n, x in a.items() if n not in LEAVES}
    ref = gdn_gradients(leaves, d_o, dh, **rest)
    compare(got, ref, a["q"].dtype, rows)
    return got


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("K,V", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("T", [1, 17, 64, 65, 200])
def test_dense(T, K, V, dtype):
    check(make(B=2, T=T, H=2, G=2, K=K, V=V, dtype=dtype, h0=T % 2 == 1, seed=T), dht=T != 64)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("lens", [[1], [63, 1, 64], [0, 130, 0, 5, 64, 0]])
def test_packed(lens, dtype):
    check(make(H=1, G=3, K=64, V=128, lens=lens, dtype=dtype, h0=True, seed=len(lens)))


# segments (dense and ragged, with sequences of one segment and of none next to long ones)
@pytest.mark.parametrize("kw", [
    dict(T=1030, G=1, K=128, V=128), dict(T=900, G=2, K=64, V=128), dict(T=770, G=2, K=128, V=64, raw=True, gate="softplus"),
    dict(lens=[900, 0, 64, 600, 1], G=1, K=64, V=64), dict(B=2, T=700, G=2, K=64, V=64)])
@pytest.mark.parametrize("h0", [False, True])
def test_segments(kw, h0):
    check(make(H=1, h0=h0, **kw), dht=h0)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("gate,dt_bias", [(None, True), ("softplus", True), ("softplus", False), ("bounded", True)])
@pytest.mark.parametrize("T", [3, 90])
def test_prestage(T, gate, dt_bias, dtype):
    check(make(B=2, T=T, H=2, G=2, K=128, V=64, dtype=dtype, raw=True, gate=gate, dt_bias=dt_bias, h0=True))


@pytest.mark.parametrize("kind", ["strong", "mixed", "none"])
def test_decays(kind):
    a = make(T=150, H=2, K=64, V=64, h0=True, seed=3)
    if kind == "strong":
        a["g"].mul_(0).sub_(40.0)
    elif kind == "mixed":
        a["g"][:, 5] = -3000.0
    else:
        a["g"].zero_()
    check(a)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_cleared_state_passes_no_gradient(dtype):
    # at g = -inf the state starts anew: nothing before it sees what follows, and nothing is NaN
    a = make(T=100, H=1, K=64, V=64, dtype=dtype, h0=True)
    a["g"][:, 70] = -torch.inf
    d_o, dh = cotangents(a)
    d_o[:, :70] = 0
    out = dict(zip(OUTS, kda.gdn_bwd(**to(a, DEV), d_o=d_o.to(DEV), dht=dh.to(DEV))))
    for n in ("q", "k", "v", "g", "beta", "initial_state"):
        assert torch.isfinite(out[n]).all(), n
        if n == "g" and dtype == FP:
            # kda_bwd's dg is a suffix sum of differences: what follows cancels to the rounding of
            # up to 128 additions, 128 x 2^-24 of the largest sum
            assert out[n][:, :70].abs().max() <= 2.0 ** -17 * out[n].abs().max()
        elif n != "initial_state":
            assert (out[n][:, :70] == 0).all(), n
    assert (out["initial_state"] == 0).all() and out["v"][:, 70:].float().norm() > 0


def test_zero_beta():
    a = make(T=100, H=2, K=64, V=64, h0=True)
    a["beta"].zero_()
    got = check(a)
    assert (got["v"] == 0).all() and got["beta"].float().norm() > 0


def test_equal_keys():
    a = make(T=130, H=1, K=64, V=64, seed=4)
    a["k"] = a["k"][:, :1].expand_as(a["k"]).contiguous()
    check(a)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_rows_behind_the_last_sequence_stay(dtype):
    a = make(lens=[70, 3], tail=90, H=2, K=64, V=64, dtype=dtype, raw=True, gate="softplus")
    d_o, dh = cotangents(a)
    plan = kda.GdnBwdPlan(**to(a, DEV), d_o=d_o.to(DEV), dht=dh.to(DEV))
    rows = (plan.dq, plan.dk, plan.dv, plan.dg, plan.dbeta)
    for x in rows:
        x.fill_(7.0)
    out = dict(zip(OUTS, plan()))
    for x in rows:
        assert (x[:, 73:] == 7.0).all()
    leaves = {n: a[n] for n in LEAVES if a.get(n) is not None}
    cut = lambda x: x[:, :73]
    leaves = {n: cut(x) if n in ("q", "k", "v", "g", "beta") else x for n, x in leaves.items()}
    rest = {n: x for n, x in a.items() if n not in LEAVES}
    compare(out, gdn_gradients(leaves, cut(d_o), dh, **rest), dtype, rows=73)


def test_no_tokens():
    a = to(make(lens=[0, 0], H=1, K=64, V=64, h0=True), DEV)
    dh = torch.randn(2, 1, 64, 64, device=DEV)
    out = kda.gdn_bwd(**a, d_o=torch.empty_like(a["v"]), dht=dh)
    assert torch.equal(out[5], dh)


def test_runs_are_equal_and_streams_do_not_matter():
    a = to(make(B=2, T=150, H=2, G=2, K=128, V=128, h0=True), DEV)
    d_o = torch.randn_like(a["v"])
    dh = torch.randn(2, 4, 128, 128, device=DEV)
    want = kda.gdn_bwd(**a, d_o=d_o, dht=dh)
    plans = [kda.GdnBwdPlan(**a, d_o=d_o, dht=dh) for _ in range(2)]
    torch.cuda.synchronize()
    for p in plans:
        p(stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    for p in plans:
        for x, y in zip(p._outs[:6], want[:6]):
            assert torch.equal(x, y)


@pytest.mark.parametrize("dtype,T", [(BF, 200), (FP, 200), (BF, 1000)])
def test_replays_of_a_graph(dtype, T):
    kw = dict(B=1, T=T, H=2, K=64, V=64, dtype=dtype, raw=True, gate="softplus", h0=True)
    a = to(make(**kw), DEV)
    d_o = torch.randn_like(a["v"])
    plan = kda.GdnBwdPlan(**a, d_o=d_o)
    plan()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan()
    for seed in range(3):
        new = to(make(**kw, seed=seed + 7), DEV)
        for n, x in a.items():
            if torch.is_tensor(x):
                x.copy_(new[n])
        want = kda.gdn_bwd(**a, d_o=d_o)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(plan._outs, want):
            assert torch.equal(x, y)


# -------------------------------------------------------------------------------- autograd

def grads(fn, a, d_o, dh, **kw):
    leaves = {n: a[n].clone().requires_grad_() for n in LEAVES if a.get(n) is not None}
    o, fin = fn(**(a | leaves), **kw)
    torch.autograd.backward([o, fin], [d_o, dh])
    return o, fin, {n: x.grad for n, x in leaves.items()}


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("checkpoint", [None, "int8"])
def test_chunk_gdn(checkpoint, dtype):
    a = to(make(B=2, T=90, H=2, G=2, K=64, V=128, dtype=dtype, raw=True, gate="softplus", h0=True), DEV)
    d_o, dh = (x.to(DEV) for x in cotangents(a))
    o, fin, got = grads(kda.chunk_gdn, a, d_o, dh, checkpoint=checkpoint)
    want_o, want_fin = kda.gdn_fwd(**a)
    assert torch.equal(o, want_o) and torch.equal(fin, want_fin)
    b = dict(a)
    if checkpoint:
        for n in ("q", "k", "v"):
            b[n] = kda.unpack8(kda.pack8(a[n]))
    want = dict(zip(OUTS, kda.gdn_bwd(**b, d_o=d_o, dht=dh)))
    for n, x in got.items():
        assert x.dtype == a[n].dtype and torch.equal(x, want[n]), n


@pytest.mark.parametrize("dtype", [BF, FP])
def test_chunk_kda_from_checkpoints(dtype):
    a = to(make(B=1, T=70, H=2, K=64, V=64, dtype=dtype, h0=True), DEV)
    a["g"] = a["g"][..., None].expand(-1, -1, -1, 64).contiguous()
    d_o, dh = (x.to(DEV) for x in cotangents(a))
    o, _, got = grads(kda.chunk_kda, a, d_o, dh, checkpoint="int8")
    plain, _, exact = grads(kda.chunk_kda, a, d_o, dh)
    assert torch.equal(o, plain)
    b = a | {n: kda.unpack8(kda.pack8(a[n])) for n in ("q", "k", "v")}
    want = dict(zip(OUTS, kda.kda_bwd(**b, d_o=d_o, dht=dh)))
    for n, x in got.items():
        assert torch.equal(x, want[n].to(a[n].dtype)), n
        # an element of a row is off by 1 / 254 of the row's largest: about 1% of the rms
        assert (x.float() - exact[n].float()).norm() <= 0.1 * exact[n].float().norm(), n


def test_packed_inputs_are_their_values():
    a = to(make(lens=[30, 0, 100], H=2, K=64, V=64), DEV)
    d_o = torch.randn_like(a["v"])
    p = {n: kda.pack8(a[n]) for n in ("q", "k", "v")}
    got = kda.gdn_bwd(**(a | p), d_o=d_o)
    want = kda.gdn_bwd(**(a | {n: kda.unpack8(x) for n, x in p.items()}), d_o=d_o)
    for x, y in zip(got[:6], want[:6]):
        assert torch.equal(x, y)


def test_long_and_short_sequences_of_many_heads():
    # each sequence by a call of its own: two results, each within its bar
    lens = [100, 4000, 1, 700, 64, 2500, 1000]
    a = to(make(lens=lens + [0], H=16, G=2, K=64, V=64, h0=True), DEV)
    d_o, dh = (x.to(DEV) for x in cotangents(a))
    got = kda.gdn_bwd(**a, d_o=d_o, dht=dh)
    at = 0
    for s, n in enumerate(lens):
        part = {m: a[m][:, at:at + n].contiguous() for m in ("q", "k", "v", "g", "beta")}
        want = kda.gdn_bwd(**part, initial_state=a["initial_state"][s:s + 1], d_o=d_o[:, at:at + n].contiguous(),
                           dht=dh[s:s + 1])
        for m, x, y in zip(OUTS[:6], got, want):
            x = x[s:s + 1] if m == "initial_state" else x[:, at:at + n]
            assert (x.double() - y.double()).norm() <= 2 * tol(m, BF) * y.double().norm(), (s, m)
        at += n
    assert torch.equal(got[5][7], dh[7])


def test_offsets_beyond_32_bits():
    # 2.2e9 elements a tensor; the last sequence by calls of its own, each result within its bar
    n, N, H, D = 33000, 8, 64, 128
    gen = torch.Generator(device=DEV).manual_seed(1)
    big = lambda *s: torch.empty(*s, dtype=BF, device=DEV).normal_(generator=gen)
    a = {m: big(1, n * N, H, D) for m in ("q", "k", "v")}
    a["g"] = -big(1, n * N, H).abs() * 0.1
    a["beta"] = big(1, n * N, H)
    d_o = big(1, n * N, H, D)
    assert d_o.numel() > 2 ** 31
    pre = dict(use_qk_l2norm=True, use_beta_sigmoid=True)
    cu = torch.arange(0, n * N + 1, n, device=DEV)
    part = {m: x[:, -n:].contiguous() for m, x in a.items()}
    far = lambda x, y: float((x.double() - y.double()).norm() / y.double().norm())
    o, fin = kda.gdn_fwd(**a, cu_seqlens=cu, **pre)
    want_o, want_fin = kda.gdn_fwd(**part, **pre)
    assert far(o[:, -n:], want_o) <= 2.0 ** -7 and far(fin[-1:], want_fin) <= 2 * 2.0 ** -13
    del o, want_o
    got = kda.gdn_bwd(**a, d_o=d_o, cu_seqlens=cu, **pre)
    want = kda.gdn_bwd(**part, d_o=d_o[:, -n:].contiguous(), **pre)
    for m, x, y in zip(OUTS[:5], got, want):
        assert far(x[:, -n:], y) <= 2 * tol(m, BF), m
    assert far(got[5][-1:], want[5]) <= 2 * tol("initial_state", BF)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_some_or_all_inputs_packed(dtype):
    a = to(make(B=2, T=77, H=2, G=2, K=64, V=128, dtype=dtype, raw=True, gate="softplus", h0=True), DEV)
    d_o, dh = (x.to(DEV) for x in cotangents(a))
    p = {n: kda.pack8(a[n]) for n in ("q", "k", "v")}
    for names in ("qkv", "qk", "v"):
        b = {n: p[n] for n in names}
        got = kda.gdn_bwd(**(a | b), d_o=d_o, dht=dh)
        want = kda.gdn_bwd(**(a | {n: kda.unpack8(x) for n, x in b.items()}), d_o=d_o, dht=dh)
        for x, y in zip(got, want):
            assert torch.equal(x, y), names


def test_replays_of_a_graph_from_checkpoints():
    a = to(make(T=150, H=2, K=64, V=64), DEV)
    d_o = torch.randn_like(a["v"])
    p = {n: kda.pack8(a[n]) for n in ("q", "k", "v")}
    plan = kda.GdnBwdPlan(**(a | p), d_o=d_o)
    plan()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan()
    for seed in range(3):
        torch.manual_seed(seed)
        for n in p:
            q = kda.pack8(torch.randn_like(a[n].float()).bfloat16() * 0.1)
            p[n].data.copy_(q.data)
            p[n].scale.copy_(q.scale)
        want = kda.gdn_bwd(**(a | p), d_o=d_o)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(plan._outs[:6], want[:6]):
            assert torch.equal(x, y)


def test_gradient_is_the_forwards_difference():
    # the GPU's own forward (fp32 io) along a direction: (f(x + e d) - f(x - e d)) / 2 e
    a = to(make(T=100, H=1, K=64, V=64, dtype=FP, h0=True, seed=9), DEV)
    d_o, dh = (x.to(DEV) for x in cotangents(a))
    _, _, got = grads(kda.chunk_gdn, a, d_o, dh)
    gen = torch.Generator(device=DEV).manual_seed(3)

    def loss(b):
        o, fin = kda.gdn_fwd(**b)
        return float((o.double() * d_o).sum() + (fin.double() * dh).sum())
    for n in ("q", "k", "v", "g", "beta", "initial_state"):
        step = torch.randn(a[n].shape, generator=gen, device=DEV)
        e = 1e-3
        diff = (loss(a | {n: a[n] + e * step}) - loss(a | {n: a[n] - e * step})) / (2 * e)
        slope = float((got[n].double() * step).sum())
        # the loss sums 6400 o and 4096 state values of about 0.1 .. 1 with fp32 errors of about
        # 1e-7: 1e-5 / 2e-3 of noise; e^2 times a third derivative of about the slope's size
        assert abs(diff - slope) <= 0.02 + 1e-3 * got[n].double().norm(), n


@pytest.mark.parametrize("checkpoint", [None, "int8"])
def test_chunk_gdn_rows_behind_the_last_sequence_are_zero(checkpoint):
    a = to(make(lens=[70, 0, 100], H=2, K=64, V=64, tail=30), DEV)
    a["v"][:, 170:] = float("nan")              # read by nothing
    d_o = torch.randn_like(a["v"].float()).bfloat16()
    poison = [torch.full_like(a[n], float("nan")) for n in ("q", "k", "v", "g", "beta") for _ in range(3)]
    del poison                                  # new tensors may well start as these
    leaves = {n: a[n].clone().requires_grad_() for n in ("q", "k", "v", "g", "beta")}
    o, _ = kda.chunk_gdn(**leaves, cu_seqlens=a["cu_seqlens"], checkpoint=checkpoint)
    o.backward(d_o)
    assert (o[:, 170:] == 0).all() and torch.isfinite(o).all()
    for n, x in leaves.items():
        assert (x.grad[:, 170:] == 0).all() and torch.isfinite(x.grad).all() and x.grad.norm() > 0, n


def test_second_derivatives_are_refused():
    a = to(make(T=20, H=1, K=64, V=64, dtype=FP), DEV)
    q = a["q"].clone().requires_grad_()
    o, _ = kda.chunk_gdn(**(a | {"q": q}))
    dq, = torch.autograd.grad(o.square().sum(), q, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        dq.sum().backward()


def test_training_step_runs():
    torch.manual_seed(0)
    a = to(make(B=2, T=70, H=2, K=64, V=64, raw=True), DEV)
    w = torch.nn.Parameter(a["q"].clone())
    o, _ = kda.chunk_gdn(**(a | {"q": w}), checkpoint="int8")
    o.sum().backward()
    assert w.grad.shape == w.shape and torch.isfinite(w.grad).all() and w.grad.float().norm() > 0
