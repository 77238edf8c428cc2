"""Long sequences of the gated linear recurrence, which tiles take that hand states to each other: against the
recurrence in 64 bits across tiles, windows of tiles and spans of windows (64 or 128 tokens, 8 tiles, 8 windows), and
what else such calls have to hold."""
from __future__ import annotations

import pytest
import torch

import chunked_kimi_delta_amd as kda
from glr_cases import check_forward, check_gradients, make, to
from oracle.glr import glr_gradients, glr_recurrent

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = [torch.bfloat16, torch.float32]
SHAPES = [dict(T=4096, D=130, h0=True), dict(T=9001, D=3), dict(B=2, T=4500, D=66, h0=True), dict(T=18000, D=2),
          dict(lens=[700, 0, 9000, 1, 2300], D=34, h0=True, tail=5), dict(lens=[8192, 128, 64, 4096], D=65),
          dict(lens=[0, 12000, 0], D=4, h0=True)]
PRE = [dict(), dict(beta=True), dict(sigmoid=True, gate="softplus"), dict(gate="bounded", dt_bias=False)]


def gradients(a, y, d_y, dht):
    b = to(a, DEV)
    return kda.glr_bwd(b.pop("x"), b.pop("g"), y, d_y, dht=dht, want_dh0="initial_state" in a, **b)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pre", PRE, ids=["plain", "beta", "softplus", "bounded"])
@pytest.mark.parametrize("kw", SHAPES, ids=lambda k: "-".join(f"{n}{v}" for n, v in k.items()))
def test_forward_and_gradients(kw, pre, dtype):
    a = make(dtype=dtype, g_lo=0.99, g_hi=0.9999, **kw, **pre)
    y, fin = kda.glr_fwd(**to(a, DEV))
    torch.cuda.synchronize()
    check_forward(a, y, fin, *glr_recurrent(**a))
    gen = torch.Generator().manual_seed(5)
    d_y = torch.randn(y.shape, generator=gen).to(dtype)
    dht = torch.randn(fin.shape, generator=gen) if "initial_state" in a else None
    rows = sum(kw["lens"]) if "lens" in kw else kw["T"]
    y[:, rows:] = 0
    got = gradients(a, y, d_y.to(DEV), None if dht is None else dht.to(DEV))
    torch.cuda.synchronize()
    check_gradients(a, y.cpu(), d_y, dht, got, glr_gradients(**a, y=y.cpu(), d_y=d_y, dht=dht))
    # the same bits again, whichever workgroups come first
    for _ in range(3):
        y2, fin2 = kda.glr_fwd(**to(a, DEV))
        again = gradients(a, y, d_y.to(DEV), None if dht is None else dht.to(DEV))
        assert torch.equal(y2[:, :rows], y[:, :rows]) and torch.equal(fin2, fin)
        for p, q in zip(got, again):
            assert p is None or (torch.equal(p[:, :rows], q[:, :rows]) if p.dim() == 3 else torch.equal(p, q))


@pytest.mark.parametrize("n", [64, 65, 150])
def test_many_packed_sequences(n):
    gen = torch.Generator().manual_seed(n)
    lens = [int(x) for x in torch.randint(900, 1400, (n,), generator=gen)]
    lens[3], lens[4] = 0, 2600
    a = make(lens=lens, D=2, h0=True, dtype=torch.float32)
    y, fin = kda.glr_fwd(**to(a, DEV))
    check_forward(a, y, fin, *glr_recurrent(**a))
    d_y = torch.randn_like(y)
    b = to(a, DEV)
    dx, dg, _, dh0, _, _ = kda.glr_bwd(b.pop("x"), b.pop("g"), y, d_y, **b)
    for s in (0, 3, 4, 62, 63, n - 1):              # each as it is alone: a batch of its own takes strips
        lo, hi = int(a["cu_seqlens"][s]), int(a["cu_seqlens"][s + 1])
        one = {m: a[m][:, lo:hi].contiguous() for m in ("x", "g")} | {"initial_state": a["initial_state"][s:s + 1]}
        part, d = y[:, lo:hi].cpu(), d_y[:, lo:hi].cpu()
        got = (dx[:, lo:hi], dg[:, lo:hi], None, dh0[s:s + 1], None, None)
        check_gradients(one, part, d, None, got, glr_gradients(**one, y=part, d_y=d))


@pytest.mark.parametrize("dtype", TYPES)
def test_slow_strong_and_clearing_decays(dtype):
    T = 20000
    g = torch.tensor([0.0, -1e-7, -1e-5, -1e-3, -0.005, -0.3, -0.51, -20.0, -float("inf"), 1e-5])
    D = len(g)
    a = dict(x=torch.ones(1, T, D).to(dtype), g=g.expand(1, T, D).contiguous().to(dtype), initial_state=torch.full((1, D), 3.0))
    a["g"][0, 1::2, 5] = -1e-4                       # both sorts of a decay in one lane
    y, fin = kda.glr_fwd(**to(a, DEV))
    check_forward(a, y, fin, *glr_recurrent(**a))
    d_y, dht = torch.ones(1, T, D).to(dtype), torch.full((1, D), 2.0)
    got = gradients(a, y, d_y.to(DEV), dht.to(DEV))
    check_gradients(a, y.cpu(), d_y, dht, got, glr_gradients(**a, y=y.cpu(), d_y=d_y, dht=dht))


def test_bad_values_stay_in_their_channel_and_sequence():
    a = make(lens=[5000, 9000, 2000], D=20, h0=True)
    b = to(a, DEV)
    y0, f0 = kda.glr_fwd(**b)
    b["x"][0, 6000, 7], b["g"][0, 6100, 9] = float("nan"), float("nan")
    y, fin = kda.glr_fwd(**b)
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[0, 6000:14000, 7] = hit[0, 6100:14000, 9] = True
    assert torch.equal(y[~hit], y0[~hit]) and torch.isnan(y[hit]).all()
    clean = torch.ones_like(fin, dtype=torch.bool)
    clean[1, 7] = clean[1, 9] = False
    assert torch.equal(fin[clean], f0[clean]) and torch.isnan(fin[~clean]).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_behind_the_last_sequence_stay(dtype):
    a = make(lens=[9000, 100], D=10, tail=300, sigmoid=True, gate="softplus", dtype=dtype)
    for n in ("x", "g", "beta"):
        a[n][:, 9100:] = float("nan")
    b = to(a, DEV)
    y = torch.full_like(b["x"], 7.0)
    kda.GlrFwdPlan(**b, y=y)()
    d_y = torch.full_like(y, float("nan"))
    d_y[:, :9100] = 1.0
    back = kda.GlrBwdPlan(b.pop("x"), b.pop("g"), y, d_y, **b)
    for t in (back.dx, back.dg, back.dbeta):
        t.fill_(7.0)
    back()
    torch.cuda.synchronize()
    for t in (y, back.dx, back.dg, back.dbeta):
        assert (t[:, 9100:] == 7).all() and torch.isfinite(t).all()
    assert torch.isfinite(back.dA_log).all() and torch.isfinite(back.ddt_bias).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [16, 9])
def test_columns_of_a_projection_and_states_in_place(D, dtype):
    a = to(make(T=5000, D=D, sigmoid=True, gate="softplus", h0=True, dtype=dtype), DEV)
    want = kda.glr_fwd(**a)
    wide = torch.cat([a["x"], a["g"], a["beta"], torch.full_like(a["x"], float("nan"))], 2)
    views = dict(zip(("x", "g", "beta"), wide.split(D, 2)))
    h = a["initial_state"].clone()
    got = kda.GlrFwdPlan(**(a | views | {"initial_state": h}), final_state=h)()
    assert torch.equal(got[0], want[0]) and torch.equal(h, want[1])
    d_y = torch.randn_like(want[0])
    rest = {n: x for n, x in a.items() if n not in ("x", "g", "beta")}
    for p, q in zip(kda.glr_bwd(a["x"], a["g"], want[0], d_y, a["beta"], **rest),
                    kda.glr_bwd(views["x"], views["g"], want[0], d_y, views["beta"], **rest)):
        assert torch.equal(p, q)


@pytest.mark.parametrize("which", ["fwd", "bwd"])
def test_replays_of_a_graph(which):
    a = to(make(lens=[5000, 0, 7000], D=70, h0=True, sigmoid=True, gate="softplus", tail=5), DEV)
    y0, _ = kda.glr_fwd(**a)
    d_y = torch.randn_like(y0)

    def call():
        if which == "fwd":
            return kda.glr_fwd(**a)
        b = dict(a)
        return kda.glr_bwd(b.pop("x"), b.pop("g"), y0, d_y, **b)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for seed in range(4):
        torch.manual_seed(seed)
        for n in ("x", "g", "beta"):
            a[n].copy_(torch.randn(a[n].shape))
        a["initial_state"].copy_(torch.randn(a["initial_state"].shape))
        a["cu_seqlens"].copy_(torch.tensor([0, 100 + 900 * seed, 9000, 12000]))
        want = [None if t is None else t.clone() for t in call()]
        for t in out:
            if t is not None:
                t.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(out, want):
            if p is not None:
                assert torch.equal(p[:, :12000], q[:, :12000]) if p.dim() == 3 else torch.equal(p, q)


def test_calls_side_by_side():
    """Two long calls on two streams at once, each with its own workspace, and a kernel that holds compute units."""
    a, b = (to(make(T=30000, D=256, h0=True, seed=s), DEV) for s in (1, 2))
    want = kda.glr_fwd(**a), kda.glr_fwd(**b)
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    w = torch.randn(4096, 4096, device=DEV)
    for _ in range(5):
        with torch.cuda.stream(one):
            p = kda.glr_fwd(**a)
        with torch.cuda.stream(two):
            q = kda.glr_fwd(**b)
        w @ w
        torch.cuda.synchronize()
        for got, ref in zip((p, q), want):
            assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_chunk_glr_of_a_long_sequence():
    a = to(make(T=6000, D=12, h0=True, sigmoid=True, gate="softplus"), DEV)
    names = ("x", "g", "beta", "initial_state", "A_log", "dt_bias")
    leaves = {n: a[n].clone().requires_grad_() for n in names}
    y, fin = kda.chunk_glr(**(a | leaves))
    d_y, dht = torch.randn_like(y), torch.randn_like(fin)
    torch.autograd.backward([y, fin], [d_y, dht])
    b = dict(a)
    ref = kda.glr_bwd(b.pop("x"), b.pop("g"), y.detach(), d_y, dht=dht, **b)
    for n, r in zip(names, ref):
        assert torch.equal(leaves[n].grad, r), n


def test_a_capture_of_the_backward_while_an_eager_graph_lives():
    a = to(make(T=4200, D=16, dtype=torch.float32), DEV)
    x, g = (a[n].clone().requires_grad_() for n in ("x", "g"))
    y, _ = kda.chunk_glr(x, g)
    y.sum().backward()
    plan = kda.GlrBwdPlan(None, g.detach(), y.detach(), torch.ones_like(y.detach()))
    plan()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan()
    for t in plan._outs[:2]:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(plan.dx, x.grad) and torch.equal(plan.dg, g.grad)
