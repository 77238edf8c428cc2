"""Pools of states on the GPU against lists in Python, exactly; then pools, steps and these calls together, as a
server runs them."""
from __future__ import annotations

import pytest
import torch

import chunked_kimi_delta_amd as kda
from gdn_cases import make as make_gdn
from gdn_cases import to

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
# slots of whole and broken 16 KiB pieces and 16-byte units, of every alignment, beside each other
LAYERS = [((4, 64, 64), torch.float32), ((777,), torch.float32), ((3,), torch.bfloat16), ((5000,), torch.bfloat16),
          ((1,), torch.int8), ((4097, 4), torch.float32), ((16384,), torch.uint8)]


def make(slots, layers=LAYERS, seed=0):
    gen = torch.Generator().manual_seed(seed)
    return [torch.randint(1, 100, (slots, *shape), generator=gen).to(dtype) for shape, dtype in layers]


def same(got, want):
    torch.cuda.synchronize()
    for i, (p, q) in enumerate(zip(got, want)):
        assert torch.equal(p.cpu(), q), i


def up(x):
    return [t.to(DEV) for t in x] if x and torch.is_tensor(x[0]) else torch.tensor(x, dtype=torch.int32, device=DEV)


def define_fork(pools, used, src, sources=None):
    dst, free = [], [i for i, u in enumerate(used) if not u]
    have = len(used) if sources is None else sources[0].shape[0]
    ok = [0 <= s < have and (sources is not None or bool(used[s])) for s in src]
    take = [p.clone() for p in (pools if sources is None else sources)]
    for s, good in zip(src, ok):
        at = free.pop(0) if good and free else -1
        dst.append(at)
        if at >= 0:
            used[at] = True
            for p, f in zip(pools, take):
                p[at] = f[s]
    return dst


def define_free(pools, used, indices):
    for i in indices:
        if 0 <= i < len(used):
            used[i] = False
            for p in pools:
                p[i] = 0


def define_compact(pools, used, indices):
    count = int(used.sum())
    holes = [i for i in range(count) if not used[i]]
    tail = [i for i in range(count, len(used)) if used[i]]
    for a, b in zip(tail, holes):
        for p in pools:
            p[b] = p[a]
            p[a] = 0
    new = dict(zip(tail, holes))
    used[:] = torch.arange(len(used)) < count
    return count, [new.get(i, i) for i in indices]


@pytest.mark.parametrize("src,dst", [([0], [5]), ([3, 3, 1], [0, 7, 6]), ([2, -1, 4, 9, 1, 0], [5, 6, 9, 7, -3, 0]), ([], [])])
def test_copy(src, dst):
    pools = make(9)
    got = up(pools)
    kda.pool_copy(got, up(src), up(dst))
    for a, b in zip(src, dst):
        if 0 <= a < 9 and 0 <= b < 9:
            for p in pools:
                p[b] = p[a]
    same(got, pools)


def test_copy_one_pool_and_sources():
    pools, others = make(6), make(4, seed=1)
    got, src = up(pools), up(others)
    kda.pool_copy(got, up([3, 0, 5, 1]), up([5, 1, 0, 2]), sources=src)
    for a, b in ((3, 5), (0, 1), (1, 2)):
        for p, q in zip(pools, others):
            p[b] = q[a]
    same(got, pools)
    kda.pool_copy(got, dst=up([2, 0, 4, 5]), sources=src)          # row i
    for a, b in enumerate((2, 0, 4, 5)):
        for p, q in zip(pools, others):
            p[b] = q[a]
    same(got, pools)
    kda.pool_copy(got, src=up([1, 1]), sources=src)                # to slot i
    for p, q in zip(pools, others):
        p[0] = p[1] = q[1]
    same(got, pools)
    kda.pool_copy(got, sources=src)                                # all of them
    for p, q in zip(pools, others):
        p[:4] = q
    same(got, pools)
    one = got[0].clone()
    kda.pool_copy(one, up([0]), up([3]))
    assert torch.equal(one[3], got[0][0]) and torch.equal(one[:3], got[0][:3])


@pytest.mark.parametrize("slots,live,src", [
    (8, [1, 2, 5], [5, 1]), (8, [0, 1, 2, 3, 4, 5, 6], [6, 0, 2]), (8, [], [0, 1]), (8, list(range(8)), [1]),
    (8, [2, 3], [2, -1, 3, 8, 2, 7, 2]), (3000, list(range(0, 3000, 2)), [-1, 4, 6] * 400 + [2998]), (5, [0], [])])
def test_fork(slots, live, src):
    layers = LAYERS if slots < 100 else LAYERS[1:3]
    pools, used = make(slots, layers), torch.zeros(slots, dtype=torch.bool)
    used[live] = True
    got, gused = up(pools), used.to(DEV)
    dst = kda.pool_fork(got, gused, up(src))
    want = define_fork(pools, used, src)
    same([dst, gused, *got], [torch.tensor(want, dtype=torch.int32), used, *pools])


def test_fork_from_sources_and_alloc():
    pools, others, used = make(7), make(3, seed=2), torch.zeros(7, dtype=torch.bool)
    used[[0, 3]] = True
    got, src, gused = up(pools), up(others), used.to(DEV)
    dst = kda.pool_fork(got, gused, sources=src)
    want = define_fork(pools, used, [0, 1, 2], others)
    same([dst, gused, *got], [torch.tensor(want, dtype=torch.int32), used, *pools])
    assert kda.pool_alloc(gused, 5).tolist() == [5, 6, -1, -1, -1] and gused.all()
    assert kda.pool_alloc(gused, 0).tolist() == []
    same(got, pools)


@pytest.mark.parametrize("indices", [[], [0], [3, 3, -1, 8, 5, 3], list(range(8))])
def test_free(indices):
    pools, used = make(8), torch.ones(8, dtype=torch.bool)
    used[6] = False
    got, gused = up(pools), used.to(DEV)
    kda.pool_free(got, gused, up(indices))
    define_free(pools, used, indices)
    same([gused, *got], [used, *pools])
    kda.pool_free((), gused, up([7, 7]))                           # no pools: only marked
    used[7] = False
    same([gused, *got], [used, *pools])


@pytest.mark.parametrize("slots,live", [(8, []), (8, [7]), (8, [0, 1, 2]), (8, [1, 2, 5, 6]), (8, list(range(8))), (1, [0]),
                                        (1025, list(range(3, 1025, 3))), (5000, list(range(2600, 5000)))])
def test_compact(slots, live):
    layers = LAYERS if slots < 100 else LAYERS[1:4]
    pools, used = make(slots, layers), torch.zeros(slots, dtype=torch.bool)
    used[live] = True
    for p in pools:
        p[~used] = 0
    indices = [-1, slots, *live[::-1], *live[:2]]                   # padding, every row, some twice
    got, gused, gi = up(pools), used.to(DEV), up(indices)
    count = kda.pool_compact(got, gused, gi)
    want, renumbered = define_compact(pools, used, indices)
    assert count.tolist() == [want] and gi.tolist() == renumbered
    same([gused, *got], [used, *pools])


def test_many_pools_in_one_call():
    layers = [((40 + i,), torch.float32) for i in range(70)]        # more than a launch takes
    pools = make(5, layers)
    got = up(pools)
    kda.pool_copy(got, up([1, 4]), up([0, 2]))
    for p in pools:
        p[0], p[2] = p[1], p[4]
    same(got, pools)


def test_pools_beyond_32_bits():
    pool = torch.zeros(9, 1 << 28, dtype=torch.float32, device=DEV)       # 1 GiB a slot
    pool[7].normal_()
    used = torch.zeros(9, dtype=torch.bool, device=DEV)
    used[7] = True
    dst = kda.pool_fork(pool, used, up([7]))
    assert dst.tolist() == [0] and torch.equal(pool[0], pool[7]) and not pool[1:7].any()
    kda.pool_copy(pool, up([0]), up([8]))
    assert torch.equal(pool[8], pool[7])
    kda.pool_free(pool, used, up([0]))
    rows = up([7])
    assert kda.pool_compact(pool, used, rows).tolist() == [1] and rows.tolist() == [0]
    assert torch.equal(pool[0], pool[8]) and not pool[7].any()


def test_bad_arguments_on_the_device():
    p, used, i = torch.zeros(8, 4, device=DEV), torch.zeros(8, dtype=torch.bool, device=DEV), up([1])
    for call in (lambda: kda.pool_copy([p, torch.zeros(7, 4, device=DEV)], i, i),
                 lambda: kda.pool_copy(p, i, up([1, 2])), lambda: kda.pool_copy(p, i, i, sources=[p, p]),
                 lambda: kda.pool_copy(p, i, i, sources=torch.zeros(8, 5, device=DEV)),
                 lambda: kda.pool_copy(torch.zeros(8, 0, device=DEV), i, i),
                 lambda: kda.pool_fork(p, used[:7], i), lambda: kda.pool_fork(p, used),
                 lambda: kda.pool_free(p, used, i.cpu()), lambda: kda.pool_alloc(used, -1)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: kda.pool_copy(p, i.long(), i), lambda: kda.pool_free(p, used.to(torch.uint8), i),
                 lambda: kda.pool_compact(p, used, i.long())):
        with pytest.raises(TypeError):
            call()


def test_replays_of_a_graph():
    pools, used = up(make(40, LAYERS[:3])), torch.zeros(40, dtype=torch.bool, device=DEV)
    rows = torch.full((20,), -1, dtype=torch.int32, device=DEV)

    def turn():
        new = kda.pool_fork(pools, used, rows[:8])
        kda.pool_free(pools, used, rows[:8])
        rows[:8] = new
        return new, kda.pool_compact(pools, used, rows)
    turn()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = turn()
    for seed in range(4):
        torch.manual_seed(seed)
        order = torch.randperm(40)[:20 + seed].to(torch.int32)
        p0, u0, r0 = make(40, LAYERS[:3], seed), torch.zeros(40, dtype=torch.bool), order[:20]
        u0[order.long()] = True

        def restore():
            for p, q in zip(pools, p0):
                p.copy_(q)
            used.copy_(u0)
            rows.copy_(r0)
        restore()
        want = [t.clone() for t in (*turn(), rows, used, *pools)]
        restore()
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip((*out, rows, used, *pools), want):
            assert torch.equal(p, q)


def test_other_streams():
    pools, used = up(make(30)), torch.zeros(30, dtype=torch.bool, device=DEV)
    used[:9] = True
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        new = kda.pool_fork(pools, used, up([8, 2]))
        kda.pool_free(pools, used, up([0]))
        count = kda.pool_compact(pools, used, new)
    side.synchronize()
    want, u = make(30), torch.zeros(30, dtype=torch.bool)
    u[:9] = True
    dst = define_fork(want, u, [8, 2])
    define_free(want, u, [0])
    n, dst = define_compact(want, u, dst)
    assert count.tolist() == [n] and new.tolist() == dst
    same([used, *pools], [u, *want])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_server_of_two_layers(dtype):
    """A delta-rule layer and a recurrence layer over one set of slots: prompts are admitted, stepped, forked,
    freed and compacted, and every row's outputs stay those of its own sequence run alone."""
    H, K, D, slots, gen = 2, 64, 48, 7, torch.Generator().manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=gen).to(dtype).to(DEV)

    def tokens(B, T):
        a = to(make_gdn(B=B, T=T, H=H, K=K, V=K, dtype=dtype, seed=int(torch.randint(1 << 20, (1,), generator=gen))), DEV)
        return a, dict(x=n(B, T, D), g=-n(B, T, D).abs())
    pools = [torch.zeros(slots, H, K, K, device=DEV), torch.zeros(slots, D, device=DEV)]
    used = torch.zeros(slots, dtype=torch.bool, device=DEV)
    a, b = tokens(3, 20)
    _, s0 = kda.gdn_fwd(**a)
    _, s1 = kda.glr_fwd(**b)
    rows = kda.pool_fork(pools, used, sources=[s0, s1])
    own = [[s0[i].clone(), s1[i].clone()] for i in range(3)]       # each row's states, kept apart
    for turn in range(4):
        a, b = tokens(len(own), 1)
        o = kda.gdn_step(**a, state=pools[0], state_indices=rows)
        y = kda.glr_step(**b, state=pools[1], state_indices=rows)
        for i, states in enumerate(own):
            s0, s1 = states[0][None].clone(), states[1][None].clone()
            oi = kda.gdn_step(**{m: t[i:i + 1].contiguous() for m, t in a.items()}, state=s0)
            yi = kda.glr_step(**{m: t[i:i + 1].contiguous() for m, t in b.items()}, state=s1)
            assert torch.equal(o[i], oi[0]) and torch.equal(y[i], yi[0]), (turn, i)
            own[i] = [s0[0], s1[0]]
        if turn == 1:                                              # row 0 twice more, row 1 gone
            new = kda.pool_fork(pools, used, rows[[0, 0]])
            kda.pool_free(pools, used, rows[1:2])
            rows = torch.cat([rows[[0, 2]], new])
            kda.pool_compact(pools, used, rows)
            own = [own[0], own[2], own[0], own[0]]
            assert sorted(rows.tolist()) == [0, 1, 2, 3] and used.tolist() == [True] * 4 + [False] * 3
            assert not pools[0][4:].any() and not pools[1][4:].any()
