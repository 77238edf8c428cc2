"""The gated linear recurrence on the GPU against its recurrence in 64 bits: forward, gradients and serving step,
at lengths around a lane's, a wave's and a workgroup's tokens, odd channel counts, views, packed batches; then the
calls' behaviour (streams, graphs, in-place states, rows that must stay, bad values)."""
from __future__ import annotations

import pytest
import torch

import chunked_kimi_delta_amd as kda
from glr_cases import check, check_forward, check_gradients, forward_bound, make, to
from oracle.glr import glr_gradients, glr_recurrent

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = [torch.bfloat16, torch.float32]

SHAPES = [dict(T=1, D=1), dict(T=7, D=2), dict(T=8, D=33), dict(T=64, D=64, h0=True), dict(B=3, T=65, D=18),
          dict(T=511, D=17, h0=True), dict(T=513, D=6), dict(B=2, T=1030, D=34, h0=True),
          dict(lens=[70, 0, 1, 513, 64], D=20, h0=True, tail=9), dict(lens=[0], D=5, h0=True, tail=3)]
PRE = [dict(), dict(beta=True), dict(sigmoid=True, gate="softplus"), dict(gate="bounded", dt_bias=False)]


def run_fwd(a, **kw):
    out = kda.glr_fwd(**to(a, DEV), **kw)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pre", PRE, ids=["plain", "beta", "softplus", "bounded"])
@pytest.mark.parametrize("kw", SHAPES, ids=lambda k: "-".join(f"{n}{v}" for n, v in k.items()))
def test_forward_and_gradients(kw, pre, dtype):
    a = make(dtype=dtype, **kw, **pre)
    y, fin = run_fwd(a)
    ref_y, ref_fin = glr_recurrent(**a)
    check_forward(a, y, fin, ref_y, ref_fin)
    gen = torch.Generator().manual_seed(5)
    d_y = torch.randn(y.shape, generator=gen).to(dtype)
    dht = torch.randn(fin.shape, generator=gen) if "initial_state" in a else None
    y = y.cpu()
    if "cu_seqlens" in a:
        y[:, int(a["cu_seqlens"][-1]):] = 0
    b = to(a, DEV)
    got = kda.glr_bwd(b.pop("x"), b.pop("g"), y.to(DEV), d_y.to(DEV), dht=None if dht is None else dht.to(DEV),
                      want_dh0="initial_state" in a, **b)
    torch.cuda.synchronize()
    check_gradients(a, y, d_y, dht, got, glr_gradients(**a, y=y, d_y=d_y, dht=dht))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [1100, 77])
def test_many_sequences_take_wide_strips(D, dtype):
    lens = [3, 70, 0, 9] * 20
    a = make(lens=lens, D=D, h0=True, beta=True, dtype=dtype)
    y, fin = run_fwd(a)
    check_forward(a, y, fin, *glr_recurrent(**a))
    gen = torch.Generator().manual_seed(6)
    d_y, dht = torch.randn(y.shape, generator=gen).to(dtype), torch.randn(fin.shape, generator=gen)
    b = to(a, DEV)
    got = kda.glr_bwd(b.pop("x"), b.pop("g"), y, d_y.to(DEV), dht=dht.to(DEV), **b)
    check_gradients(a, y.cpu(), d_y, dht, got, glr_gradients(**a, y=y.cpu(), d_y=d_y, dht=dht))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kw", [dict(B=2, T=40, D=12), dict(lens=[33, 5], D=9, tail=2)])
def test_columns_of_a_projection(kw, dtype):
    a = make(sigmoid=True, gate="softplus", h0=True, dtype=dtype, **kw)
    D = a["x"].shape[2]
    want = run_fwd(a)
    wide = torch.cat([a["x"], a["g"], a["beta"], torch.full_like(a["x"], float("nan"))], 2).to(DEV)
    views = dict(zip(("x", "g", "beta"), wide.split(D, 2)))
    got = kda.glr_fwd(**(to(a, DEV) | views))
    rows = sum(kw["lens"]) if "lens" in kw else kw["T"]
    assert torch.equal(got[0][:, :rows], want[0][:, :rows]) and torch.equal(got[1], want[1])
    d_y = torch.randn_like(want[0])
    b = to(a, DEV)
    rest = {n: x for n, x in b.items() if n not in ("x", "g", "beta")}
    g1 = kda.glr_bwd(b["x"], b["g"], want[0], d_y, b["beta"], **rest)
    g2 = kda.glr_bwd(views["x"], views["g"], want[0], d_y, views["beta"], **rest)
    for p, q in zip(g1, g2):
        assert torch.equal(p[:, :rows], q[:, :rows]) if p.dim() == 3 else torch.equal(p, q)
    if "B" in kw:
        step = [kda.glr_step(v["x"], v["g"], b["initial_state"].clone(), v["beta"], **{n: x for n, x in rest.items() if n != "initial_state"})
                for v in (b, views)]
        assert torch.equal(*step)


def test_backward_takes_y_and_its_gradient_as_views():
    a = to(make(B=3, T=37, D=10, dtype=torch.float32), DEV)
    y, _ = kda.glr_fwd(**a)
    d_y = torch.randn_like(y)
    padded = lambda t: torch.cat([t, torch.full_like(t[:, :5], float("nan"))], 1)[:, :37]
    want = kda.glr_bwd(None, a["g"], y, d_y)
    for p, q in zip(kda.glr_bwd(None, a["g"], padded(y), padded(d_y)), want):
        assert p is None or torch.equal(p, q)
    ones = torch.ones((), device=DEV).expand(3, 37, 10)             # what the gradient of a sum is
    for p, q in zip(kda.glr_bwd(None, a["g"], y, ones), kda.glr_bwd(None, a["g"], y, torch.ones_like(y))):
        assert p is None or torch.equal(p, q)


def test_strides_that_are_refused():
    x = torch.zeros(2, 6, 8, device=DEV)
    for bad in (x.transpose(1, 2)[:, :6, :6], x[:, ::2][:, :, :6].transpose(0, 1), x[:, :, ::2], x[:1].expand(2, 6, 8)):
        good = torch.zeros(bad.shape, device=DEV)
        with pytest.raises(ValueError, match="evenly spaced"):
            kda.glr_fwd(bad, good)
        with pytest.raises(ValueError, match="evenly spaced"):
            kda.glr_fwd(good, bad)
    kda.glr_fwd(x[:, :, :3], x[:, :, 3:6])
    kda.glr_fwd(x[:, :1], x[:, 3:4])
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", TYPES)
def test_strong_slow_and_clearing_decays(dtype):
    """Decays of every size, one a channel, -inf among them; and slow ones, whose distance from 1 counts."""
    T, D = 700, 12
    g = torch.tensor([0.0, -1e-6, -1e-5, -1e-4, -1e-2, -0.3, -0.49, -0.51, -3.0, -20.0, -80.0, -float("inf")]).expand(1, T, D)
    a = dict(x=torch.ones(1, T, D).to(dtype), g=g.contiguous().to(dtype), initial_state=torch.full((1, D), 3.0))
    y, fin = run_fwd(a)
    ref_y, ref_fin = glr_recurrent(**a)
    check_forward(a, y, fin, ref_y, ref_fin)
    # nothing but a first value: what a strong decay leaves, to |g| 2^-23 of itself a token (fp32 holds 2^-126)
    a["x"] = torch.zeros_like(a["x"])
    y, fin = run_fwd(a)
    ref_y, ref_fin = glr_recurrent(**a)
    t = torch.arange(1, T + 1, dtype=torch.float64)[None, :, None]
    size = a["g"].double().abs().clamp_max(200.0)
    tol = (2.0 ** -8 if dtype == torch.bfloat16 else 0.0) + t * (size + 4) * 2.0 ** -22
    assert ((y.cpu().double() - ref_y).abs() <= tol * ref_y.abs() + 2.0 ** -120).all()
    assert ((fin.cpu().double() - ref_fin).abs() <= tol[:, -1] * ref_fin.abs() + 2.0 ** -120).all()


def test_bad_values_stay_in_their_channel_and_sequence():
    a = make(lens=[100, 600, 50], D=40, h0=True, beta=True)
    y0, f0 = run_fwd(a)
    a["x"] = a["x"].clone()
    a["x"][0, 300, 7], a["x"][0, 310, 9] = float("nan"), float("inf")
    y, fin = run_fwd(a)
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[0, 300:700, 7] = hit[0, 310:700, 9] = True
    assert torch.equal(y[~hit], y0[~hit]) and not torch.isfinite(y[hit]).any()
    clean = torch.ones_like(fin, dtype=torch.bool)
    clean[1, 7] = clean[1, 9] = False
    assert torch.equal(fin[clean], f0[clean])


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_behind_the_last_sequence_stay(dtype):
    a = make(lens=[20, 5], D=10, tail=7, beta=True, gate="softplus", dtype=dtype)
    for n in ("x", "g", "beta"):
        a[n][:, 25:] = float("nan")
    b = to(a, DEV)
    y = torch.full_like(b["x"], 7.0)
    plan = kda.GlrFwdPlan(**b, y=y)
    plan()
    d_y = torch.full_like(y, float("nan"))
    d_y[:, :25] = 1.0
    back = kda.GlrBwdPlan(b.pop("x"), b.pop("g"), y, d_y, **b)
    for t in (back.dx, back.dg, back.dbeta):
        t.fill_(7.0)
    back()
    torch.cuda.synchronize()
    for t in (y, back.dx, back.dg, back.dbeta):
        assert (t[:, 25:] == 7).all() and torch.isfinite(t).all()
    assert torch.isfinite(back.dA_log).all() and torch.isfinite(back.ddt_bias).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_state_in_place_and_pieces(dtype):
    a = make(T=900, D=24, h0=True, beta=True, dtype=dtype)
    y, fin = run_fwd(a)
    b = to(a, DEV)
    h = b["initial_state"]
    whole = kda.GlrFwdPlan(**b, final_state=h)()
    assert torch.equal(whole[0], y) and torch.equal(h, fin)
    h = to(a, DEV)["initial_state"]                 # the same in pieces, each from the one before
    parts = []
    for lo, hi in ((0, 1), (1, 333), (333, 333), (333, 900)):
        c = {n: b[n][:, lo:hi] for n in ("x", "g", "beta")}
        part, h = kda.glr_fwd(**c, initial_state=h)
        parts.append(part)
    by, bf = forward_bound(a)
    check(torch.cat(parts, 1), y.double().cpu(), 2 * by + (2.0 ** -8 * y.abs().double().cpu() if dtype == torch.bfloat16 else 0), dtype, "y")
    check(h, fin.double().cpu(), 2 * bf, torch.float32, "state")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pre", PRE, ids=["plain", "beta", "softplus", "bounded"])
@pytest.mark.parametrize("B,T,D", [(1, 1, 1), (5, 1, 34), (3, 4, 7), (9, 3, 600)])
def test_step(B, T, D, pre, dtype):
    a = make(B=B, T=T, D=D, dtype=dtype, **pre)
    pool = torch.randn(B + 3, D)
    at = torch.randperm(B + 3)[:B].to(torch.int32)
    if B > 2:
        at[1], at[2] = -1, B + 3                    # padding of both kinds
    live = (at >= 0) & (at < B + 3)
    state = pool.to(DEV)
    y = kda.glr_step(**to(a, DEV), state=state, state_indices=at.to(DEV))
    torch.cuda.synchronize()
    h0 = pool[at.long().clamp(0, B + 2)]
    ref_y, ref = glr_recurrent(**a, initial_state=h0)
    by, bf = forward_bound(a | {"initial_state": h0})
    check(y[live.to(DEV)], ref_y[live], by[live], dtype, "y")
    assert (y[~live.to(DEV)] == 0).all()
    check(state[at[live].long().to(DEV)], ref[live], bf[live], torch.float32, "state")
    rest = torch.ones(B + 3, dtype=torch.bool)
    rest[at[live].long()] = False
    assert torch.equal(state.cpu()[rest], pool[rest])
    state = pool.to(DEV)                            # no indices: row b in slot b
    kda.glr_step(**to(a, DEV), state=state)
    check(state[:B], glr_recurrent(**a, initial_state=pool[:B])[1], forward_bound(a | {"initial_state": pool[:B]})[1],
          torch.float32, "state")
    assert torch.equal(state[B:].cpu(), pool[B:])


@pytest.mark.parametrize("kw", [dict(T=70, D=9), dict(lens=[40, 0, 30], D=8, tail=6)])
@pytest.mark.parametrize("dtype", TYPES)
def test_chunk_glr(kw, dtype):
    a = to(make(h0=True, sigmoid=True, gate="softplus", dtype=dtype, **kw), DEV)
    names = ("x", "g", "beta", "initial_state", "A_log", "dt_bias")
    leaves = {n: a[n].clone().requires_grad_() for n in names}
    if "lens" in kw:
        for n in ("x", "g", "beta"):
            leaves[n].data[:, 70:] = float("nan")
    y, fin = kda.chunk_glr(**(a | leaves))
    d_y, dht = torch.randn_like(y), torch.randn_like(fin)
    (y.float() * d_y.float()).sum().backward(retain_graph=True)
    for x in leaves.values():
        x.grad = None
    torch.autograd.backward([y, fin], [d_y, dht])
    b = dict(a)
    ref = kda.glr_bwd(b.pop("x"), b.pop("g"), y.detach(), d_y, dht=dht, **b)
    for n, r in zip(("x", "g", "beta", "initial_state", "A_log", "dt_bias"), ref):
        got = leaves[n].grad
        if r.dim() == 3:
            assert torch.equal(got[:, :70], r[:, :70]) and (got[:, 70:] == 0).all(), n
        else:
            assert torch.equal(got, r), n
    assert (y[:, 70:] == 0).all()
    y, _ = kda.chunk_glr(**(a | leaves))
    (gx,) = torch.autograd.grad(y.float()[:, :70].square().sum(), [leaves["x"]], create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        gx.float().sum().backward()


def test_gradients_against_differences():
    a = to(make(T=300, D=6, h0=True, sigmoid=True, gate="softplus", dtype=torch.float32), DEV)
    names = ("x", "g", "beta", "initial_state", "A_log", "dt_bias")
    leaves = {n: a[n].clone().requires_grad_() for n in names}
    y, fin = kda.chunk_glr(**(a | leaves))
    d_y, dht = torch.randn_like(y), torch.randn_like(fin)
    torch.autograd.backward([y, fin], [d_y, dht])

    def loss(b):
        y, fin = kda.glr_fwd(**b)
        return float((y.double() * d_y).sum() + (fin.double() * dht).sum())
    for n in names:
        step = torch.randn_like(a[n])
        e = 2.0 ** -7
        diff = (loss(a | {n: a[n] + e * step}) - loss(a | {n: a[n] - e * step})) / (2 * e)
        want = float((leaves[n].grad.double() * step).sum())
        # fp32 outputs: the loss errs by about 2^-24 sqrt(1800) of its terms (some tens) over 2 e, and the
        # differences by e^2 / 6 of a third derivative a few times the first: 6e-5, taken thrice as a bound
        size = float((leaves[n].grad.double() * step).norm())
        assert abs(diff - want) <= 2e-4 * abs(want) + 1e-3 * size + 2e-2, n


def test_gradients_of_bf16_through_the_forward():
    """dg takes the states from y as rounded: against autograd in 64 bits, half a step of y more."""
    a = make(T=200, D=16, h0=True)
    y, _ = run_fwd(a)
    d_y = torch.randn(y.shape).bfloat16()
    b = to(a, DEV)
    got = kda.glr_bwd(b.pop("x"), b.pop("g"), y, d_y.to(DEV), **b)
    exact_y, _ = glr_recurrent(**a)
    ref = glr_gradients(**a, y=exact_y, d_y=d_y)
    err = (got[1].double().cpu() - ref["g"]).abs()
    # half a step of y, half a step of dg, and both the forward's and the backward's own errors
    m = ref["g"].abs()
    by, _ = forward_bound(a)
    slack = 2.0 ** -13 * (ref["dh"].abs() + 1) * (exact_y.abs() + 1)
    assert (err <= (2 * 2.0 ** -8 + 2.0 ** -16) * m + slack).all()


@pytest.mark.parametrize("which", ["fwd", "bwd", "step"])
def test_replays_of_a_graph(which):
    shape = dict(B=3, T=2, D=64, sigmoid=True, gate="softplus") if which == "step" else dict(
        lens=[1200, 0, 77], D=64, h0=True, sigmoid=True, gate="softplus", tail=5)
    a = to(make(**shape), DEV)
    state = torch.randn(5, 64, device=DEV)
    index = torch.tensor([4, -1, 0], dtype=torch.int32, device=DEV)
    y0, _ = kda.glr_fwd(**a)
    d_y = torch.randn_like(y0)

    def call():
        if which == "fwd":
            return kda.glr_fwd(**a)
        if which == "step":
            return kda.glr_step(**a, state=state, state_indices=index), state
        b = dict(a)
        return kda.glr_bwd(b.pop("x"), b.pop("g"), y0, d_y, **b)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for seed in range(3):
        torch.manual_seed(seed)
        for n in ("x", "g", "beta"):
            a[n].copy_(torch.randn(a[n].shape))
        keep = torch.randn_like(state)
        if "initial_state" in a:
            a["initial_state"].copy_(torch.randn(a["initial_state"].shape))
            a["cu_seqlens"].copy_(torch.tensor([0, 100 + seed, 1000, 1277]))
        state.copy_(keep)
        want = [None if t is None else t.clone() for t in call()]
        state.copy_(keep)
        for t in out:
            if t is not None and t is not state:
                t.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(out, want):
            if p is not None:
                assert torch.equal(p[:, :1277], q[:, :1277]) if p.dim() == 3 else torch.equal(p, q)


def test_other_streams_and_repeats_agree():
    a = to(make(B=2, T=2000, D=96, h0=True, sigmoid=True, gate="bounded"), DEV)
    want = kda.glr_fwd(**a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = kda.glr_fwd(**a)
    plan = kda.GlrFwdPlan(**a)
    other = [t.clone() for t in plan(side)]
    side.synchronize()
    for p, q, r in zip(want, got, plan(side)):
        side.synchronize()
        assert torch.equal(p, q) and torch.equal(p, r)


@pytest.mark.parametrize("gate", [None, "softplus"])
def test_no_tokens(gate):
    a = to(make(B=2, T=3, D=5, h0=True, sigmoid=True, gate=gate), DEV)
    a |= {n: a[n][:, :0] for n in ("x", "g", "beta")}
    y, fin = kda.glr_fwd(**a)
    assert y.shape == (2, 0, 5) and torch.equal(fin, a["initial_state"])
    dht = torch.randn_like(fin)
    b = dict(a)
    dx, dg, db, dh0, dA, ddt = kda.glr_bwd(b.pop("x"), b.pop("g"), y, y.clone(), dht=dht, **b)
    assert torch.equal(dh0, dht) and dx.shape == dg.shape == db.shape == (2, 0, 5)
    assert gate is None or (not dA.any() and not ddt.any())
    state = torch.randn(2, 5, device=DEV)
    keep = state.clone()
    b = {n: x for n, x in a.items() if n != "initial_state"}
    assert kda.glr_step(**b, state=state).shape == (2, 0, 5) and torch.equal(state, keep)


def test_sequences_of_a_batch_are_what_they_are_alone():
    """The same sequence alone (narrow strips) and among many (wide strips): the bounds of two evaluations."""
    lens = [900] + [40] * 60
    a = make(lens=lens, D=640, h0=True, dtype=torch.float32)
    y, fin = run_fwd(a)
    one = dict(x=a["x"][:, :900], g=a["g"][:, :900], initial_state=a["initial_state"][:1])
    y1, f1 = run_fwd({n: t.contiguous() for n, t in one.items()})
    by, bf = forward_bound(one)
    check(y[:, :900], y1.double().cpu(), 2 * by, torch.float32, "y")
    check(fin[:1], f1.double().cpu(), 2 * bf, torch.float32, "state")


def test_rows_beyond_32_bits():
    """More than 2^32 bytes in a tensor and sequence: the last rows against a call of their own."""
    T, D = (1 << 20) + 77, 2050
    x = torch.empty(1, T, D, dtype=torch.bfloat16, device=DEV).normal_()
    g = torch.full((1, T, D), -0.25, dtype=torch.bfloat16, device=DEV)
    y, fin = kda.glr_fwd(x, g)
    tail = slice(T - 700, T)                        # 600 tokens at -0.25 leave e^-150 of what was before
    y1, f1 = kda.glr_fwd(x[:, tail].contiguous(), g[:, tail].contiguous())
    assert (y[:, -100:].float() - y1[:, -100:].float()).abs().max() <= 2.0 ** -7 * 8
    assert (fin - f1).abs().max() <= 1e-4
    dx, dg, *_ = kda.glr_bwd(None, g, y, x)
    head = slice(0, 700)
    dx1, dg1, *_ = kda.glr_bwd(None, g[:, head].contiguous(), y[:, head].contiguous(), x[:, head].contiguous())
    assert (dx[:, :100].float() - dx1[:, :100].float()).abs().max() <= 2.0 ** -7 * 8
    assert (dg[:, :100].float() - dg1[:, :100].float()).abs().max() <= 2.0 ** -7 * 64
