"""The gated delta rule on the GPU against the fp64 token recurrence (oracle/gdn.py): every type,
head dim and grouping, lengths around a chunk's 64 tokens, packed and empty sequences, strong
decays, the pre-stage, and the serving step over a pool of states."""
from __future__ import annotations

import pytest
import torch

import chunked_kimi_delta_amd as kda
from errlog import report_named
from gdn_cases import check_o, check_state, make, to
from oracle.gdn import gdn_recurrent

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, FP = torch.bfloat16, torch.float32


def run(a, **kw):
    out = kda.gdn_fwd(**to(a, DEV), **kw)
    torch.cuda.synchronize()
    return out


def check(a, rows=None):
    dt = a["q"].dtype
    o, fin = run(a)
    ref, rfin = gdn_recurrent(**a)
    rel = lambda x, y: float((x.double().cpu() - y).norm() / y.norm().clamp_min(1e-30))
    report_named(o=rel(o, ref), final=rel(fin, rfin))
    check_o(o, ref, dt, rows)
    check_state(fin, rfin, dt)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("K,V", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("T", [1, 16, 17, 64, 65, 200])
def test_dense(T, K, V, dtype):
    check(make(B=2, T=T, H=2, G=2, K=K, V=V, dtype=dtype, h0=T % 2 == 1, seed=T))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("lens", [[1], [63, 1, 64], [0, 130, 0, 5, 64, 0], [70] * 9])
def test_packed(lens, dtype):
    check(make(H=1, G=3, K=64, V=128, lens=lens, dtype=dtype, h0=True, seed=len(lens)))


# long sequences of few heads run in segments that are joined: dense and ragged, with sequences of one
# segment and of none next to long ones
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("kw", [
    dict(T=1030, K=128, V=128), dict(T=2100, K=64, V=128), dict(T=1500, K=128, V=64, raw=True, gate="softplus"),
    dict(lens=[900, 0, 64, 1300, 1], K=64, V=64), dict(lens=[3000, 5], K=64, V=64), dict(B=2, T=700, K=64, V=64)])
def test_segments(kw, dtype):
    for h0 in (False, True):
        check(make(H=1, G=2, dtype=dtype, h0=h0, **kw))


# many heads, so that only the length beyond the mean is cut
@pytest.mark.parametrize("lens", [[100, 4000, 1, 700, 64, 0, 2500, 1000], [1200, 1000, 1100, 1024, 1088, 1, 1500, 1600]])
def test_long_and_short_sequences_of_many_heads(lens):
    check(make(lens=lens, H=32, K=64, V=64, h0=True))


def test_segments_update_the_state_in_place():
    a = to(make(T=2000, H=1, G=2, K=64, V=128, h0=True), DEV)
    o, fin = kda.gdn_fwd(**a)
    h = a["initial_state"].clone()
    o2, _ = kda.GdnFwdPlan(**(a | {"initial_state": h}), final_state=h)()
    assert torch.equal(o, o2) and torch.equal(h, fin)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("gate,dt_bias", [(None, True), ("softplus", True), ("softplus", False), ("bounded", True)])
@pytest.mark.parametrize("T", [3, 90])
def test_prestage(T, gate, dt_bias, dtype):
    check(make(B=2, T=T, H=2, G=2, K=128, V=64, dtype=dtype, raw=True, gate=gate, dt_bias=dt_bias, h0=True))


@pytest.mark.parametrize("T", [8, 150])
@pytest.mark.parametrize("kind", ["clears", "strong", "mixed", "none"])
def test_decays(kind, T):
    a = make(T=T, H=2, K=64, V=64, dtype=FP, h0=True, seed=3)
    g = a["g"]
    if kind == "clears":            # -inf: the state starts anew at these tokens
        g[:, 2::37] = -torch.inf
    elif kind == "strong":
        g.mul_(0).sub_(40.0)
    elif kind == "mixed":           # one huge decay, then slow ones: differences of large sums
        g[:, 5] = -3000.0
    else:
        g.zero_()
    check(a)


@pytest.mark.parametrize("T", [12, 130])
def test_equal_keys_and_unit_beta(T):
    # the hardest inverse: every key the same, nothing decays, beta 1 (bidiagonal inverse)
    a = make(T=T, H=1, K=64, V=64, dtype=FP, seed=4)
    a["k"] = a["k"][:, :1].expand_as(a["k"]).contiguous()
    a["g"].zero_()
    a["beta"].fill_(1.0)
    check(a)


def test_zero_beta_keeps_the_state():
    a = make(T=100, H=1, K=64, V=64, h0=True)
    a["beta"].zero_()
    a["g"].zero_()
    _, fin = run(a)
    assert torch.equal(fin.cpu(), a["initial_state"])


def test_rows_behind_the_last_sequence_stay():
    a = make(lens=[70, 3], tail=90, H=2, K=64, V=64)
    o = torch.full_like(a["v"], 7.0).to(DEV)
    plan = kda.GdnFwdPlan(**to(a, DEV), o=o)
    plan()
    ref, _ = gdn_recurrent(**a)
    check_o(o, ref, BF, rows=73)
    assert (o[:, 73:] == 7.0).all()


def test_no_tokens():
    a = make(lens=[0, 0], H=1, K=64, V=64, h0=True)
    o, fin = run(a)
    assert o.shape[1] == 0 and torch.equal(fin.cpu(), a["initial_state"])
    a = make(B=3, T=0, H=1, K=64, V=64, h0=True)
    assert torch.equal(run(a)[1].cpu(), a["initial_state"])


@pytest.mark.parametrize("T", [5, 150])
def test_state_in_place_and_without_final_state(T):
    a = to(make(B=2, T=T, H=1, G=2, K=64, V=64, h0=True), DEV)
    o, fin = kda.gdn_fwd(**a)
    o2, none = kda.gdn_fwd(**a, output_final_state=False)
    assert none is None and torch.equal(o, o2)
    h = a["initial_state"].clone()
    o3, _ = kda.GdnFwdPlan(**(a | {"initial_state": h}), final_state=h)()
    assert torch.equal(o, o3) and torch.equal(h, fin)


def test_a_nan_stays_in_its_sequence_and_head():
    a = make(lens=[100, 80, 90], H=2, K=64, V=64)
    clean, _ = run(a)
    a["v"][0, 130, 1] = torch.nan
    o, fin = run(a)
    keep = torch.ones(270, 2, dtype=torch.bool)
    keep[100:180, 1] = False
    assert torch.equal(o[0].cpu()[keep], clean[0].cpu()[keep])
    assert torch.isnan(o[0, 130:180, 1].float()).any() and torch.isfinite(fin[[0, 2]]).all()


def test_grouped_heads_are_repeated_heads_and_packed_is_dense():
    a = make(B=3, T=130, H=2, G=3, K=128, V=128, seed=6)
    o, fin = run(a)
    rep = dict(a)
    rep["q"], rep["k"] = (a[n].repeat_interleave(3, 2) for n in ("q", "k"))
    o2, fin2 = run(rep)
    assert torch.equal(o, o2) and torch.equal(fin, fin2)
    flat = {n: x.reshape(1, -1, *x.shape[2:]) for n, x in a.items()}
    o3, fin3 = run(flat | {"cu_seqlens": torch.arange(4) * 130})
    assert torch.equal(o.reshape(o3.shape), o3) and torch.equal(fin, fin3)


@pytest.mark.parametrize("K", [64, 128])
def test_many_dense_sequences(K):
    # enough of them for 128 columns a workgroup: the same sums, so what packing gives, and the oracle's
    a = make(B=5, T=150, H=32, K=K, V=128, h0=True, raw=True, gate="softplus")
    check(a)
    a = to(a, DEV)
    o, fin = kda.gdn_fwd(**a)
    flat = {n: a[n].flatten(0, 1)[None] for n in ("q", "k", "v", "g", "beta")}
    o2, fin2 = kda.gdn_fwd(**(a | flat), cu_seqlens=torch.arange(0, 751, 150, device=DEV))
    assert torch.equal(o.flatten(0, 1), o2[0]) and torch.equal(fin, fin2)


def test_equals_kda_with_the_decay_repeated():
    a = make(B=1, T=100, H=2, K=64, V=64, dtype=FP, h0=True)
    o, fin = run(a)
    b = to(a, DEV)
    b["g"] = b["g"][..., None].expand(-1, -1, -1, 64).contiguous()
    o2, fin2 = kda.kda_fwd(**b)
    # kda_fwd's own bar for fp32 io
    assert (o - o2).norm() <= 1e-4 * o2.norm() and (fin - fin2).norm() <= 1e-4 * fin2.norm()


# ------------------------------------------------------------------------------------- step

def step_case(B, T, H, G, K, V, dtype, slots, index, seed=0, **kw):
    a = make(B=B, T=T, H=H, G=G, K=K, V=V, dtype=dtype, seed=seed, **kw)
    gen = torch.Generator().manual_seed(seed + 99)
    state = 0.3 * torch.randn(slots, H * G, K, V, generator=gen)
    return a, state, None if index is None else torch.tensor(index, dtype=torch.int32)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("K,V", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("T", [1, 3])
@pytest.mark.parametrize("index,slots", [(None, 4), ([5, 0, 2, 6], 7), ([-1, 3, 9, 1], 4), ([-1] * 4, 2)])
def test_step(index, slots, T, K, V, dtype):
    a, state, at = step_case(4, T, 2, 2, K, V, dtype, slots, index, raw=True, gate="softplus")
    s = state.clone().to(DEV)
    o = kda.gdn_step(**to(a, DEV), state=s, state_indices=None if at is None else at.to(DEV))
    torch.cuda.synchronize()
    idx = list(range(4)) if at is None else at.tolist()
    live = [b for b in range(4) if 0 <= idx[b] < slots]
    want = state.double()
    for b in range(4):
        if b not in live:
            assert (o[b] == 0).all()
    if live:
        rows = {n: x[live] if torch.is_tensor(x) and n not in ("A_log", "dt_bias") else x for n, x in a.items()}
        ref, fin = gdn_recurrent(**rows, initial_state=state[[idx[b] for b in live]])
        check_o(o[live], ref, dtype)
        for n, b in enumerate(live):
            want[idx[b]] = fin[n]
    untouched = [i for i in range(slots) if i not in [idx[b] for b in live]]
    assert torch.equal(s.cpu()[untouched], state[untouched])
    # the recurrence is fp32 throughout, whatever the io type
    check_state(s, want, FP)


def test_prefill_then_steps_equal_the_whole_sequence():
    a = make(T=80, H=2, G=2, K=64, V=64, dtype=FP, h0=True, seed=8)
    d = to(a, DEV)
    part = lambda x, i, j: x[:, i:j].contiguous()
    seq = ("q", "k", "v", "g", "beta")
    o0, fin = kda.gdn_fwd(**{n: part(d[n], 0, 70) for n in seq}, initial_state=d["initial_state"])
    outs = [o0]
    for t in range(70, 80):
        outs.append(kda.gdn_step(**{n: part(d[n], t, t + 1) for n in seq}, state=fin))
    ref, rfin = gdn_recurrent(**a)
    check_o(torch.cat(outs, 1), ref, FP)
    check_state(fin, rfin, FP)


def test_many_rows_of_a_step():
    a, state, _ = step_case(70000, 1, 1, 1, 64, 64, BF, 3, None)
    at = torch.full((70000,), -1, dtype=torch.int32)
    at[65534], at[65535], at[69999] = 2, 0, 1
    s = state.to(DEV)
    o = kda.gdn_step(**to(a, DEV), state=s, state_indices=at.to(DEV))
    live = [65534, 65535, 69999]
    rows = {n: x[live] for n, x in a.items()}
    ref, fin = gdn_recurrent(**rows, initial_state=state[[2, 0, 1]])
    check_o(o[live], ref, BF)
    check_state(s[[2, 0, 1]], fin, FP)
    assert o.float().abs().sum() == o[live].float().abs().sum()


# ------------------------------------------------------------------------- streams and graphs

@pytest.mark.parametrize("T", [300, 1200])
def test_replays_of_a_graph(T):
    a = to(make(B=1, T=T, H=2, K=128, V=128, h0=True), DEV)
    st = to(make(B=2, T=1, H=2, K=128, V=128), DEV)
    pool = torch.zeros(2, 2, 128, 128, device=DEV)
    plan, step = kda.GdnFwdPlan(**a), kda.GdnStepPlan(**st, state=pool)
    plan(), step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan()
        step()
    for seed in range(3):
        for d, n in ((a, dict(B=1, T=T, h0=True)), (st, dict(B=2, T=1))):
            new = to(make(H=2, K=128, V=128, seed=seed + 20, **n), DEV)
            for x in d:
                d[x].copy_(new[x])
        pool.fill_(0.1 * seed)
        want, ws = kda.gdn_fwd(**a), pool.clone()
        wo = kda.gdn_step(**st, state=ws)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(plan.o, want[0]) and torch.equal(plan.final_state, want[1])
        assert torch.equal(step.o, wo) and torch.equal(pool, ws)


def test_other_streams():
    a = to(make(B=2, T=150, H=2, K=64, V=64, h0=True), DEV)
    want = kda.gdn_fwd(**a)
    plans = [kda.GdnFwdPlan(**a) for _ in range(3)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in plans]
    for p, s in zip(plans, streams):
        p(stream=s)
    torch.cuda.synchronize()
    for p in plans:
        assert torch.equal(p.o, want[0]) and torch.equal(p.final_state, want[1])
