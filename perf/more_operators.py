"""The gated linear recurrence (one state a channel) and the pools of states that serving steps
read: the calls that are measured, and each operator in its plain form.

For every sequence and channel, a state h that starts at h0 or zero:

    h <- e^{g_t} h + beta_t x_t;   y_t = h

Operators (a case's "op"):
  fwd   the scan over whole sequences, dense or packed: y and the final state
  bwd   the gradients of all inputs of fwd, from y as the forward returned it
  step  a serving step: new tokens of some sequences, whose states lie in a pool of slots and
        are updated in place; rows without a slot (index -1) are padding and come out as zero
  copy  slots of the pools of several layers copied to other slots
  turn  what a server does to its pools between two steps: some rows are forked into free slots, the
        slots that they came from are freed (cleared), and the live slots move to the front
"""
import math

import torch

own = False


# ------------------------------------------------------------------------------------- cases

def _glr(op, name=None, **kw):
    c = {"op": op, "B": 1, "T": 64, "lens": "", "D": 128, "dtype": "bf16", "raw": False, "h0": False}
    c.update(kw)
    if name:
        c["name"] = name
    return c


def _step(name=None, **kw):
    c = {"op": "step", "B": 1, "T": 1, "D": 128, "dtype": "bf16", "raw": True, "slots": 1, "pad": 0}
    c.update(kw)
    if name:
        c["name"] = name
    return c


def _pool(op, name=None, **kw):
    c = {"op": op, "layers": 1, "slots": 4, "live": 2, "n": 1, "heads": 1, "K": 64, "V": 64, "D": 0}
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # the second part of a short prompt, from the first one's state: latency counts
        _glr("fwd", "fwd_short_t70", T=70, D=256, raw=True, h0=True),
        # full-precision activations, an odd number of channels, a length that is no multiple
        _glr("fwd", "fwd_fp32_t1000", B=2, T=1000, D=777, dtype="fp32"),
        # eight prompts of very different lengths packed along one token axis, raw projections
        _glr("fwd", "fwd_packed8_d4096", T=21412, lens="4096,256,1040,8192,777,2048,3,5000", D=4096,
             raw=True, h0=True),
        # one layer over one very long document
        _glr("fwd", "fwd_long_t131072", T=131072, D=2048),
        # one layer's gradients in training
        _glr("bwd", "bwd_t4096_d2048", T=4096, D=2048),
        # gradients over ragged packed samples in full precision, one of them empty
        _glr("bwd", "bwd_fp32_packed5", T=708, lens="513,64,0,130,1", D=512, raw=True, h0=True, dtype="fp32"),
        # one user's next token
        _step("step_b1_d2048", D=2048, slots=4),
        # the next token of a full serving batch, eight of its rows padding
        _step("step_b64_d4096", B=64, D=4096, slots=80, pad=8),
        # one sequence's states of two small layers kept aside
        _pool("copy", "copy_1_of_8", layers=2, slots=8, n=1, heads=4),
        # half of a full batch's states copied, one layer of matrix states and one of channel states
        _pool("copy", "copy_40_of_80", slots=80, n=40, heads=32, K=128, V=128, D=4096),
        # one of six rows forked
        _pool("turn", "turn_1_of_6", layers=2, slots=8, live=6, n=1, heads=4),
        # a quarter of a batch forked
        _pool("turn", "turn_16_of_64", slots=80, live=64, n=16, heads=32, K=128, V=128, D=4096),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "fwd", "bwd", "bwd", "step", "copy", "turn"])
    if op in ("copy", "turn"):
        heads, K, V = rng.choice([1, 2, 4, 8, 16, 32]), rng.choice([64, 128]), rng.choice([64, 128])
        slots = _log_int(rng, 4, min(200, (80 << 19) // (heads * K * V)))
        live = rng.randint(2, slots - 1)
        n = rng.randint(1, slots // 2) if op == "copy" else rng.randint(1, min(live, slots - live))
        layers = rng.randint(1, max(1, min(3, (80 << 19) // (heads * K * V * slots))))
        return _pool(op, layers=layers, slots=slots, live=live, n=n, heads=heads, K=K, V=V,
                     D=rng.choice([0, 1, 7, 64, 777, 2048, 4096]))
    D = rng.choice([64, 128, 256, 777, 1000, 2048, 4096, _log_int(rng, 1, 4096)])
    if op == "step":
        B = _log_int(rng, 1, 64)
        return _step(B=B, T=rng.choice([1, 1, 1, 2, 4, 7]), D=D, slots=B + rng.randint(0, 17),
                     pad=rng.randint(0, B // 3), dtype=rng.choice(["bf16", "bf16", "fp32"]), raw=rng.random() < 0.7)
    kw = dict(D=D, raw=rng.random() < 0.5, h0=rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "bf16", "fp32"]))
    most = min(131072, (1 << (26 if op == "fwd" else 25)) // D)  # tokens in all
    if rng.random() < 0.5:
        B = rng.choice([1, 1, 2, 3, 8])
        return _glr(op, B=B, T=_log_int(rng, 1, max(2, most // B)), **kw)
    n, most = rng.randint(1, 9), min(most, 32768)
    lens = [0 if rng.random() < 0.08 else _log_int(rng, 1, max(2, most // n)) for _ in range(n)]
    lens[0] = max(lens[0], 1)
    return _glr(op, T=sum(lens), lens=",".join(map(str, lens)), **kw)


def _lengths(case):
    return [int(x) for x in case["lens"].split(",")] if case.get("lens") else [case["T"]] * case["B"]


# ------------------------------------------------------------------------------------ inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = torch.float32 if case.get("dtype") == "fp32" else torch.bfloat16

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    if case["op"] in ("copy", "turn"):
        return _prepare_pool(case, gen, dev, normal)
    B, T, D, raw = case["B"], case["T"], case["D"], case["raw"]
    s = {"op": case["op"], "raw": raw, "beta": None, "A_log": None, "dt_bias": None}
    s["x"] = normal(B, T, D).to(dt)
    if raw:  # raw projections: the call activates the decay and takes beta as logits
        s["g"], s["beta"] = (normal(B, T, D) - 1).to(dt), normal(B, T, D).to(dt)
        s["A_log"] = torch.log(0.5 + 1.5 * torch.rand(D, generator=gen, device=dev))
        s["dt_bias"] = 0.5 * normal(D)
    else:
        s["g"] = torch.log(0.9 + 0.0999 * torch.rand(B, T, D, generator=gen, device=dev)).to(dt)
    if case["op"] == "step":
        s["state"] = normal(case["slots"], D)
        at = torch.randperm(case["slots"], generator=gen, device=dev)[:B].to(torch.int32)
        at[B - case["pad"]:] = -1
        s["slots"] = at
        return s
    lens = _lengths(case)
    s["longest"], N = max(lens), len(lens)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    s["cu"] = torch.tensor(cu, dtype=torch.int64, device=dev) if case.get("lens") else None
    s["h0"] = normal(N, D) if case["h0"] else None
    if case["op"] == "bwd":
        s["d_y"] = normal(B, T, D).to(dt)
        s["dht"] = normal(N, D) if case["h0"] else None
        s["y"] = _plain_fwd(s)[0]  # what the forward pass has returned
    return s


def _prepare_pool(case, gen, dev, normal):
    slots, n = case["slots"], case["n"]
    shapes = [(slots, case["heads"], case["K"], case["V"])] * case["layers"]
    if case["D"]:
        shapes.append((slots, case["D"]))
    s = {"op": case["op"], "pools": [normal(*x) for x in shapes]}
    order = torch.randperm(slots, generator=gen, device=dev).to(torch.int32)
    if case["op"] == "copy":
        s["src"], s["dst"] = order[:n].clone(), order[n:2 * n].clone()
        return s
    s["n"], live = n, order[:case["live"]]
    s["rows"] = live.clone()  # the slot of each row in flight
    s["used"] = torch.zeros(slots, dtype=torch.bool, device=dev)
    s["used"][live.long()] = True
    for p in s["pools"]:  # free slots are clear
        p[~s["used"]] = 0
    return s


# --------------------------------------------------------------------------------- plain forms

def _active(s):
    """log decay and input gate as the recurrence takes them, in 32 bits (beta None: one)."""
    g, beta = s["g"].float(), None if s["beta"] is None else torch.sigmoid(s["beta"].float())
    if s["raw"]:
        u = g + s["dt_bias"]
        g = -torch.exp(s["A_log"]) * (u.clamp_min(0) + torch.log1p(torch.exp(-u.abs())))
    return g, beta


def _lay(s, x):
    """Every sequence's rows, zeros behind its end: [N, longest, D]."""
    if s["cu"] is None:
        return x
    at = torch.arange(s["longest"], device=x.device)
    first, length = s["cu"][:-1], s["cu"][1:] - s["cu"][:-1]
    live = at < length[:, None]
    return x[0][torch.where(live, first[:, None] + at, 0)] * live[..., None].to(x.dtype)


def _back(s, x, like):
    if s["cu"] is None:
        return x
    at = torch.arange(s["longest"], device=x.device)
    first, length = s["cu"][:-1], s["cu"][1:] - s["cu"][:-1]
    live = at < length[:, None]
    out = x.new_zeros(like.shape)
    out[0, (first[:, None] + at)[live]] = x[live]
    return out


def _scan(a, x, h):
    """h_t = a_t h_{t-1} + x_t along dim 1 from h [N, D]: all h_t, and the last."""
    N, T, D = x.shape
    C = 1 << max(0, (T.bit_length() + 1) // 2)
    n = -(-T // C)
    a = torch.nn.functional.pad(a, (0, 0, 0, n * C - T), value=1.0).reshape(N, n, C, D)
    x = torch.nn.functional.pad(x, (0, 0, 0, n * C - T)).reshape(N, n, C, D)
    local, decay = torch.empty_like(x), torch.empty_like(x)
    p, q = torch.zeros_like(x[:, :, 0]), torch.ones_like(x[:, :, 0])
    for t in range(C):  # every chunk from a zero state
        p, q = a[:, :, t] * p + x[:, :, t], a[:, :, t] * q
        local[:, :, t], decay[:, :, t] = p, q
    starts = torch.empty_like(p)
    for c in range(n):  # the state that each chunk starts from
        starts[:, c] = h
        h = q[:, c] * h + p[:, c]
    return (local + decay * starts[:, :, None]).reshape(N, n * C, D)[:, :T], h


def _first(s, x):
    return x.new_zeros(x.shape[0], x.shape[2]) if s["h0"] is None else s["h0"]


def _plain_fwd(s):
    g, beta = _active(s)
    x = s["x"].float() if beta is None else s["x"].float() * beta
    g, x = _lay(s, g), _lay(s, x)
    y, h = _scan(torch.exp(g), x, _first(s, x))
    return _back(s, y, s["x"]).to(s["x"].dtype), h


def _plain_bwd(s):
    g, beta = _active(s)
    dt = s["x"].dtype
    gl, dy, y = _lay(s, g), _lay(s, s["d_y"].float()), _lay(s, s["y"].float())
    a, h0 = torch.exp(gl), _first(s, dy)
    last = torch.zeros_like(h0) if s["dht"] is None else s["dht"]
    # backwards in time: dh_t = dy_t + a_{t+1} dh_{t+1}. Behind a sequence's end a is one and dy zero,
    # so that the gradient of the final state arrives there unchanged.
    after = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    dh = _scan(after.flip(1), dy.flip(1), last)[0].flip(1)
    before = torch.cat([h0[:, None], y[:, :-1]], 1)
    dg = _back(s, a * before * dh, s["x"])
    dh0 = a[:, 0] * dh[:, 0]
    if s["cu"] is not None:
        dh0 = torch.where((s["cu"][1:] > s["cu"][:-1])[:, None], dh0, last)
    dh = _back(s, dh, s["x"])
    out = {"dx": dh if beta is None else beta * dh}
    if s["raw"]:
        out["dbeta"] = s["x"].float() * dh * beta * (1 - beta)
        du = -dg * torch.exp(s["A_log"]) * torch.sigmoid(s["g"].float() + s["dt_bias"])
        out["dA_log"] = (dg * g).sum((0, 1), dtype=torch.float64)
        out["ddt_bias"] = du.sum((0, 1), dtype=torch.float64)
        dg = du
    out["dg"] = dg
    if s["h0"] is not None:
        out["dh0"] = dh0
    return {n: x.to(dt) if x.dim() == 3 else x.float() for n, x in out.items()}


def _plain_step(s):
    g, beta = _active(s)
    a, x = torch.exp(g), s["x"].float() if beta is None else s["x"].float() * beta
    live = s["slots"] >= 0
    at = torch.where(live, s["slots"], 0).long()
    h, y = s["state"][at], torch.zeros_like(x)
    for t in range(x.shape[1]):
        h = a[:, t] * h + x[:, t]
        y[:, t] = h
    s["state"][at[live]] = h[live]
    return (y * live[:, None, None]).to(s["x"].dtype), s["state"]


def _plain_turn(s):
    pools, used, rows, n = s["pools"], s["used"], s["rows"], s["n"]
    old = rows[:n].long()
    new = torch.nonzero(~used)[:n, 0]  # the lowest free slots
    for p in pools:
        p[new] = p[old]
        p[old] = 0
    used[new] = True
    used[old] = False
    rows[:n] = new.to(torch.int32)
    count = used.sum().to(torch.int32)
    at = torch.arange(used.numel(), device=used.device)
    holes = torch.nonzero(~used & (at < count))[:, 0]
    tail = torch.nonzero(used & (at >= count))[:, 0]
    for p in pools:
        p[holes] = p[tail]
        p[tail] = 0
    place = at.clone()
    place[tail] = holes
    rows.copy_(place[rows.long()])
    used.copy_(at < count)
    return {"count": count.reshape(1), "rows": rows, "used": used, "pools": pools}


# ----------------------------------------------------------------------------------- one pass

def run(s):
    if not own:
        if s["op"] == "fwd":
            return _plain_fwd(s)
        if s["op"] == "bwd":
            return _plain_bwd(s)
        if s["op"] == "step":
            return _plain_step(s)
        if s["op"] == "turn":
            return _plain_turn(s)
        for p in s["pools"]:
            p[s["dst"].long()] = p[s["src"].long()]
        return s["pools"]
    import chunked_kimi_delta_amd as kda
    if s["op"] == "copy":
        kda.pool_copy(s["pools"], s["src"], s["dst"])
        return s["pools"]
    if s["op"] == "turn":
        rows, n = s["rows"], s["n"]
        new = kda.pool_fork(s["pools"], s["used"], rows[:n])
        kda.pool_free(s["pools"], s["used"], rows[:n])
        rows[:n] = new
        count = kda.pool_compact(s["pools"], s["used"], rows)
        return {"count": count, "rows": rows, "used": s["used"], "pools": s["pools"]}
    raw = dict(beta=s["beta"], use_beta_sigmoid=s["raw"], gate="softplus" if s["raw"] else None,
               A_log=s["A_log"], dt_bias=s["dt_bias"])
    if s["op"] == "step":
        y = kda.glr_step(s["x"], s["g"], s["state"], state_indices=s["slots"], **raw)
        return y, s["state"]
    if s["op"] == "fwd":
        return kda.glr_fwd(s["x"], s["g"], cu_seqlens=s["cu"], initial_state=s["h0"], **raw)
    grads = kda.glr_bwd(s["x"], s["g"], s["y"], s["d_y"], dht=s["dht"], cu_seqlens=s["cu"],
                        initial_state=s["h0"], want_dh0=s["h0"] is not None, **raw)
    return {n: x for n, x in zip(("dx", "dg", "dbeta", "dh0", "dA_log", "ddt_bias"), grads) if x is not None}


# ------------------------------------------------------------------------------------- floors

def work(case):
    if case["op"] in ("copy", "turn"):
        slot = 4 * (case["layers"] * case["heads"] * case["K"] * case["V"] + case["D"])
        # copied: read and written. A turn: forked and cleared; the rows of the holes read, moved, and cleared
        return {"bytes": case["n"] * slot * (2 if case["op"] == "copy" else 6), "flops": 0}
    e, D, raw = 4 if case["dtype"] == "fp32" else 2, case["D"], case["raw"]
    gate = 8 * D if raw else 0
    if case["op"] == "step":
        live, tokens = case["B"] - case["pad"], case["B"] * case["T"]
        return {"bytes": 8 * live * D + e * tokens * D * (4 if raw else 3) + gate, "flops": 2 * live * case["T"] * D}
    lens = _lengths(case)
    values, states = sum(lens) * D, 4 * len(lens) * D
    if case["op"] == "fwd":
        return {"bytes": e * values * (4 if raw else 3) + states * (2 if case["h0"] else 1) + gate,
                "flops": values * (3 if raw else 2)}
    return {"bytes": e * values * (8 if raw else 5) + states * (3 if case["h0"] else 0) + 2 * gate,
            "flops": values * (12 if raw else 4)}


# ------------------------------------------------------------------------------ in 64 bits

def _exact_pool(case, s):
    pools = [p.double() for p in s["pools"]]
    if case["op"] == "copy":
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            for p in pools:
                p[b] = p[a]
        return pools
    rows, used = s["rows"].tolist(), s["used"].tolist()
    old = rows[:case["n"]]
    for i, source in enumerate(old):
        rows[i] = at = used.index(False)
        used[at] = True
        for p in pools:
            p[at] = p[source]
    for at in old:
        used[at] = False
        for p in pools:
            p[at] = 0
    count = sum(used)
    for at in range(count, len(used)):
        if used[at]:
            hole = used.index(False)
            used[hole], used[at] = True, False
            rows = [hole if r == at else r for r in rows]
            for p in pools:
                p[hole] = p[at]
                p[at] = 0
    dev = s["used"].device
    return {"count": torch.tensor([count], dtype=torch.int32, device=dev),
            "rows": torch.tensor(rows, dtype=torch.int32, device=dev),
            "used": torch.tensor(used, device=dev), "pools": pools}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("copy", "turn"):
        return _exact_pool(case, s)
    x, g = s["x"].double(), s["g"].double()
    A = u = b = None
    if case["raw"]:
        A, u = s["A_log"].double().exp(), g + s["dt_bias"].double()
        g = -A * torch.nn.functional.softplus(u, threshold=1e9)
        b = 1 / (1 + torch.exp(-s["beta"].double()))
    a, w = torch.exp(g), x if b is None else b * x
    if case["op"] == "step":
        at, y = s["slots"].tolist(), torch.zeros_like(x)
        pool = s["state"].double()
        for i, slot in enumerate(at):
            for t in range(case["T"] if slot >= 0 else 0):
                pool[slot] = a[i, t] * pool[slot] + w[i, t]
                y[i, t] = pool[slot]
        return y, pool
    B, T, D = x.shape
    if s["cu"] is None:
        batches = [(0, T)]  # all rows of a batch at once, token by token
        rows, N = [slice(0, B)], B
    else:
        cu = s["cu"].tolist()
        N = len(cu) - 1
        batches, rows = [(cu[i], cu[i + 1]) for i in range(N)], [slice(0, 1)] * N
    h0 = torch.zeros(N, D, dtype=torch.float64, device=x.device) if s["h0"] is None else s["h0"].double()
    if case["op"] == "fwd":
        y, last = torch.zeros_like(x), h0.clone()
        for i, ((lo, hi), r) in enumerate(zip(batches, rows)):
            which = slice(None) if s["cu"] is None else slice(i, i + 1)
            h = h0[which]
            for t in range(lo, hi):
                h = torch.addcmul(w[r, t], a[r, t], h, out=y[r, t])
            last[which] = h
        return y, last
    y, dy = s["y"].double(), s["d_y"].double()
    dh, before = torch.zeros_like(x), torch.zeros_like(x)
    dh0 = torch.zeros_like(h0)
    for i, ((lo, hi), r) in enumerate(zip(batches, rows)):
        which = slice(None) if s["cu"] is None else slice(i, i + 1)
        d = torch.zeros_like(h0[which]) if s["dht"] is None else s["dht"].double()[which]
        if hi > lo:
            before[r, lo + 1:hi], before[r, lo] = y[r, lo:hi - 1], h0[which]
        for t in reversed(range(lo, hi)):
            dh[r, t] = dy[r, t] + d
            d = a[r, t] * dh[r, t]
        dh0[which] = d
    dg = a * before * dh
    out = {"dx": dh if b is None else b * dh}
    if case["raw"]:
        out["dbeta"] = x * dh * b * (1 - b)
        du = -A * dg / (1 + torch.exp(-u))
        out["dA_log"], out["ddt_bias"] = (dg * g).sum((0, 1)), du.sum((0, 1))
        dg = du
    out["dg"] = dg
    if s["h0"] is not None:
        out["dh0"] = dh0
    return out
