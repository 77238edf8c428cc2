"""The gated delta rule (one decay per token and value head) and its 8-bit activation
checkpoints: the calls that are measured, and each operator in its plain form.

For every sequence and value head j, with q/k head h = j / (HV / H), a state S in R^{K x V}:

    S <- e^{g_t} S;   r = v_t - S^T k_t;   S <- S + beta_t k_t r^T;   o_t = scale S^T q_t

Operators (a case's "op"):
  fwd   the forward over whole sequences, dense or packed: o and the final state
  step  a serving step: new tokens of some sequences, whose states lie in a pool of slots and
        are updated in place; rows without a slot (index -1) are padding and come out as zero
  bwd   the gradients of all inputs of fwd
  ckpt  rows of activations packed to 8 bits (one scale a row) and read back
  bwd8  bwd from q, k, v kept as 8-bit checkpoints
"""
import math

import torch

own = False

C = 64  # tokens a chunk of the plain form


# ------------------------------------------------------------------------------------- cases

def _gdn(op, name=None, **kw):
    c = {"op": op, "B": 1, "T": 64, "lens": "", "H": 1, "G": 1, "K": 128, "V": 128,
         "dtype": "bf16", "raw": False, "h0": False}
    c.update(kw)
    if name:
        c["name"] = name
    return c


def _step(name=None, **kw):
    c = {"op": "step", "B": 1, "T": 1, "H": 1, "G": 1, "K": 128, "V": 128, "dtype": "bf16",
         "raw": True, "slots": 1, "pad": 0}
    c.update(kw)
    if name:
        c["name"] = name
    return c


def _ckpt(name=None, **kw):
    c = {"op": "ckpt", "tokens": 1, "heads": 1, "D": 128, "dtype": "bf16"}
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # the second part of a short prompt, from the first one's state: latency counts
        _gdn("fwd", "fwd_short_t70", T=70, H=2, G=2, K=64, V=64, raw=True, h0=True),
        # one layer of a 4096-token training sequence or prompt
        _gdn("fwd", "fwd_h16_t4096", T=4096, H=16),
        # eight prompts of very different lengths packed along one token axis, raw projections
        _gdn("fwd", "fwd_packed8_h32", T=21412, lens="4096,256,1040,8192,777,2048,3,5000", H=32,
             raw=True, h0=True),
        # full-precision activations, key and value dims that differ, a length that is no multiple
        _gdn("fwd", "fwd_fp32_t1000", B=2, T=1000, H=4, G=2, V=64, dtype="fp32"),
        # one user's next token
        _step("step_b1_h16", H=16, slots=4),
        # the next token of a full serving batch, eight of its rows padding
        _step("step_b64_h32", B=64, H=32, slots=80, pad=8),
        # one layer's gradients in training
        _gdn("bwd", "bwd_h16_t4096", T=4096, H=16),
        # gradients over ragged packed samples in full precision, one of them empty
        _gdn("bwd", "bwd_fp32_packed5", T=708, lens="513,64,0,130,1", H=2, G=2, K=64, raw=True,
             h0=True, dtype="fp32"),
        # a short sample's activations kept for its backward pass
        _ckpt("ckpt_t333", tokens=333, heads=4, D=64),
        # q, k and v of one layer kept for the backward pass
        _ckpt("ckpt_t4096", tokens=4096, heads=48),
        # one layer's gradients from checkpoints, grouped value heads
        _gdn("bwd8", "bwd8_h8_t4096", T=4096, H=8, G=2),
        # the same for two short samples
        _gdn("bwd8", "bwd8_b2_t100", B=2, T=100, H=2, K=64, V=64, raw=True, h0=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "step", "bwd", "bwd", "ckpt", "bwd8"])
    if op == "ckpt":
        return _ckpt(tokens=_log_int(rng, 1, 8192), heads=rng.choice([1, 3, 8, 16, 24]),
                     D=rng.choice([64, 128]), dtype=rng.choice(["bf16", "bf16", "fp32"]))
    H, G = rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 1, 2, 3, 4])
    heads = dict(H=H, G=G, K=rng.choice([64, 128]), V=rng.choice([64, 128]),
                 raw=rng.random() < 0.5)
    if op == "step":
        B = _log_int(rng, 1, 48)
        return _step(B=B, T=rng.choice([1, 1, 1, 2, 4, 7]), slots=B + rng.randint(0, 17),
                     pad=rng.randint(0, B // 3), dtype=rng.choice(["bf16", "bf16", "fp32"]),
                     **heads)
    heads["dtype"] = "bf16" if op == "bwd8" else rng.choice(["bf16", "bf16", "bf16", "fp32"])
    heads["h0"] = rng.random() < 0.5
    most = (1 << 18 if op == "fwd" else 1 << 16) // (H * G)  # token-heads, below the largest listed
    if rng.random() < 0.5:
        B = rng.choice([1, 1, 2, 3])
        return _gdn(op, B=B, T=_log_int(rng, 1, min(8192, most // B)), **heads)
    n, most = rng.randint(1, 9), min(most, 16384)
    lens = [0 if rng.random() < 0.08 else _log_int(rng, 1, max(1, most // n)) for _ in range(n)]
    lens[0] = max(lens[0], 1)
    return _gdn(op, T=sum(lens), lens=",".join(map(str, lens)), **heads)


def _lengths(case):
    return [int(x) for x in case["lens"].split(",")] if case.get("lens") else [case["T"]] * case["B"]


# ------------------------------------------------------------------------------------ inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    if case["op"] == "ckpt":
        # rows whose sizes differ, as the tokens of a sequence do
        x = normal(case["tokens"], case["heads"], case["D"])
        x = x * torch.exp(normal(case["tokens"], case["heads"], 1))
        return {"op": "ckpt", "x": x.to(dt)}
    B, T, H, K, V = case["B"], case["T"], case["H"], case["K"], case["V"]
    HV = H * case["G"]
    s = {"op": case["op"], "raw": case["raw"], "gate": False, "A_log": None, "dt_bias": None}
    q, k = normal(B, T, H, K), normal(B, T, H, K)
    v, b = normal(B, T, HV, V), normal(B, T, HV)
    if case["raw"]:  # raw projections: the call normalises q and k and takes beta as logits
        q, k = 2 * q, 2 * k
    else:
        q = q * torch.rsqrt((q * q).sum(-1, keepdim=True) + 1e-6)
        k = k * torch.rsqrt((k * k).sum(-1, keepdim=True) + 1e-6)
        b = torch.sigmoid(b)
    if case["raw"] and case["op"] in ("fwd", "step"):  # and activates the decay as well
        s["gate"] = True
        g = normal(B, T, HV) - 1
        s["A_log"] = torch.log(0.5 + 1.5 * torch.rand(HV, generator=gen, device=dev))
        s["dt_bias"] = 0.5 * normal(HV)
    else:
        g = torch.log(0.9 + 0.099 * torch.rand(B, T, HV, generator=gen, device=dev))
    s.update(q=q.to(dt), k=k.to(dt), v=v.to(dt), g=g.to(dt), beta=b.to(dt))
    if case["op"] == "step":
        s["state"] = 0.1 * normal(case["slots"], HV, K, V)
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
    s["h0"] = 0.1 * normal(N, HV, K, V) if case["h0"] else None
    if case["op"] in ("bwd", "bwd8"):
        s["d_o"] = normal(B, T, HV, V).to(dt)
        s["dht"] = normal(N, HV, K, V) if case["h0"] else None
    if case["op"] == "bwd8":  # what the forward pass has kept: whole numbers and a scale a row
        for n in ("q", "k", "v"):
            s[n] = _pack(s[n])
    return s


# --------------------------------------------------------------------------------- plain forms

def _pack(x):
    """Each row as whole numbers in [-127, 127] and the scale that they count."""
    y = x.double()
    most = y.abs().amax(-1, keepdim=True)
    n = torch.where(most > 0, torch.round(y * 127 / torch.where(most > 0, most, 1.0)), 0.0)
    return n.to(torch.int8), (most / 127).float().squeeze(-1)


def _unpack(data, scale, dtype):
    return (data.float() * scale[..., None]).to(dtype)


def _norm(x):
    return torch.rsqrt((x * x).sum(-1, keepdim=True) + 1e-6)


def _active(s, q, k, g, beta):
    """q, k, g, beta as the recurrence takes them, in 32 bits."""
    q, k, g, beta = q.float(), k.float(), g.float(), beta.float()
    if s["raw"]:
        q, k, beta = q * _norm(q), k * _norm(k), torch.sigmoid(beta)
    if s["gate"]:
        x = g + s["dt_bias"]
        g = -torch.exp(s["A_log"]) * (x.clamp_min(0) + torch.log1p(torch.exp(-x.abs())))
    return q, k, g, beta


class _Chunks:
    """The sequences laid out as [N, HV, chunks, C, ...], rows past an end zero."""

    def __init__(self, s, B, T, G, dev):
        self.G, self.B, self.T = G, B, T
        self.n = -(-s["longest"] // C)
        at = torch.arange(self.n * C, device=dev)
        if s["cu"] is None:
            self.N = B
            first = torch.arange(B, device=dev) * T
            length = torch.full((B,), T, device=dev)
        else:
            self.N = s["cu"].numel() - 1
            first, length = s["cu"][:-1], s["cu"][1:] - s["cu"][:-1]
        self.live = at < length[:, None]
        self.at = torch.where(self.live, first[:, None] + at, 0)

    def lay(self, x):
        heads = x.shape[2]
        rest = x.shape[3:]
        x = x.reshape(self.B * self.T, heads, *rest)[self.at]
        x = x * self.live.reshape(self.N, -1, *[1] * (x.dim() - 2)).to(x.dtype)
        return x.transpose(1, 2).reshape(self.N, heads, self.n, C, *rest)

    def spread(self, x):  # a q/k head for each of its value heads
        return x.repeat_interleave(self.G, 1)

    def back(self, x):
        x = x.reshape(x.shape[0], x.shape[1], self.n * C, *x.shape[4:]).transpose(1, 2)
        out = x.new_zeros(self.B * self.T, *x.shape[2:])
        out[self.at[self.live]] = x[self.live]
        return out.reshape(self.B, self.T, *x.shape[2:])


def _local(q, k, v, g, beta, scale):
    """What a chunk has without its state: decays, the two triangular products, the inverse."""
    sums = torch.cumsum(g.double(), -1)
    low = torch.ones(C, C, dtype=torch.bool, device=g.device).tril()
    decay = torch.exp((sums[..., :, None] - sums[..., None, :]).masked_fill(~low, -math.inf)).float()
    head, tail = torch.exp(sums).float()[..., None], torch.exp(sums[..., -1:] - sums).float()[..., None]
    whole = torch.exp(sums[..., -1]).float()[..., None, None]
    lower = (beta[..., None] * decay * (k @ k.transpose(-1, -2))).tril(-1)
    attn = scale * decay * (q @ k.transpose(-1, -2))
    inv = torch.eye(C, device=g.device).expand_as(lower).contiguous()
    for i in range(1, C):  # forward substitution
        inv[..., i, :i] = -(lower[..., i, None, :i] @ inv[..., :i, :i])[..., 0, :]
    return decay, head, tail, whole, lower, attn, inv


def _plain_fwd(s):
    q, k, g, beta = _active(s, s["q"], s["k"], s["g"], s["beta"])
    B, T, H, K = q.shape
    HV, V = s["v"].shape[2:]
    lay = _Chunks(s, B, T, HV // H, q.device)
    scale = K ** -0.5
    q, k = lay.spread(lay.lay(q)), lay.spread(lay.lay(k))
    v, g, beta = lay.lay(s["v"].float()), lay.lay(g), lay.lay(beta)
    _, head, tail, whole, _, attn, inv = _local(q, k, v, g, beta, scale)
    inv = inv * beta[..., None, :]
    u, w, qd, kt = inv @ v, inv @ (head * k), scale * head * q, (tail * k).transpose(-1, -2)
    S = torch.zeros(lay.N, HV, K, V, device=q.device) if s["h0"] is None else s["h0"]
    o = torch.empty_like(v)
    for c in range(lay.n):
        d = u[:, :, c] - w[:, :, c] @ S
        o[:, :, c] = qd[:, :, c] @ S + attn[:, :, c] @ d
        S = whole[:, :, c] * S + kt[:, :, c] @ d
    return lay.back(o).to(s["v"].dtype), S


def _norm_back(x, dy):
    """The gradient at x of x / sqrt(sum x^2 + 1e-6)."""
    r = _norm(x)
    return r * (dy - r * r * x * (x * dy).sum(-1, keepdim=True))


def _plain_bwd(s, rq, rk, rv):
    dt, d_o = s["d_o"].dtype, s["d_o"].float()
    q, k, g, beta = _active(s, rq, rk, s["g"], s["beta"])
    B, T, H, K = q.shape
    HV, V = rv.shape[2:]
    G = HV // H
    lay = _Chunks(s, B, T, G, q.device)
    scale, b_act = K ** -0.5, beta
    q, k = lay.spread(lay.lay(q)), lay.spread(lay.lay(k))
    v, g, beta, d_o = lay.lay(rv.float()), lay.lay(g), lay.lay(beta), lay.lay(d_o)
    decay, head, tail, whole, lower, attn, inv = _local(q, k, v, g, beta, scale)
    b = beta[..., None]
    hk, tk, hq = head * k, tail * k, scale * head * q
    zero = torch.zeros(lay.N, HV, K, V, device=q.device)
    S = [zero if s["h0"] is None else s["h0"]]  # the state that each chunk starts from
    for c in range(lay.n):
        d = inv[:, :, c] @ (b[:, :, c] * (v[:, :, c] - hk[:, :, c] @ S[-1]))
        S.append(whole[:, :, c] * S[-1] + tk[:, :, c].transpose(-1, -2) @ d)
    S = torch.stack(S[:-1], 2)
    dS = [zero if s["dht"] is None else s["dht"]]  # the gradient of the state that each ends with
    for c in reversed(range(lay.n)):
        dd = attn[:, :, c].transpose(-1, -2) @ d_o[:, :, c] + tk[:, :, c] @ dS[-1]
        dr = b[:, :, c] * (inv[:, :, c].transpose(-1, -2) @ dd)
        dS.append(whole[:, :, c] * dS[-1] + hq[:, :, c].transpose(-1, -2) @ d_o[:, :, c]
                  - hk[:, :, c].transpose(-1, -2) @ dr)
    dh0 = dS.pop()
    dS = torch.stack(dS[::-1], 2)
    St, dSt = S.transpose(-1, -2), dS.transpose(-1, -2)
    r = v - hk @ S
    d = inv @ (b * r)
    dy = inv.transpose(-1, -2) @ (attn.transpose(-1, -2) @ d_o + tk @ dS)
    dr = b * dy
    d_low, d_attn = -(dy @ d.transpose(-1, -2)).tril(-1), (d_o @ d.transpose(-1, -2)).tril()
    gram, qk = d_low * b * decay, d_attn * scale * decay
    dq = qk @ k + scale * head * (d_o @ St)
    dk = (qk.transpose(-1, -2) @ q + (gram + gram.transpose(-1, -2)) @ k - head * (dr @ St)
          + tail * (d @ dSt))
    dbeta = (dy * r).sum(-1) + (d_low * decay * (k @ k.transpose(-1, -2))).sum(-1)
    pair = d_attn * attn + d_low * lower
    left = (d * (tk @ dS)).sum(-1)
    dsum = (pair.sum(-1) - pair.sum(-2) + (d_o * (hq @ S)).sum(-1) - (dr * (hk @ S)).sum(-1) - left)
    dsum[..., -1] += left.sum(-1) + whole[..., 0, 0] * (S * dS).sum((-1, -2))
    dg = dsum.flip(-1).cumsum(-1).flip(-1)
    shared = lambda x: x.unflatten(1, (H, G)).sum(2)
    dq, dk = lay.back(shared(dq)), lay.back(shared(dk))
    dv, dg, dbeta = lay.back(dr), lay.back(dg), lay.back(dbeta)
    if s["raw"]:
        dq, dk = _norm_back(rq.float(), dq), _norm_back(rk.float(), dk)
        dbeta = dbeta * b_act * (1 - b_act)
    out = {"dq": dq, "dk": dk, "dv": dv, "dg": dg, "dbeta": dbeta}
    return {n: x.to(dt) for n, x in out.items()} | ({} if s["h0"] is None else {"dh0": dh0})


def _plain_step(s):
    q, k, g, beta = _active(s, s["q"], s["k"], s["g"], s["beta"])
    G, scale = s["v"].shape[2] // q.shape[2], q.shape[3] ** -0.5
    q, k, v = q.repeat_interleave(G, 2), k.repeat_interleave(G, 2), s["v"].float()
    live = s["slots"] >= 0
    at = torch.where(live, s["slots"], 0).long()
    S, o = s["state"][at], torch.zeros_like(v)
    for t in range(q.shape[1]):
        S = torch.exp(g[:, t])[..., None, None] * S
        r = v[:, t] - (S * k[:, t, :, :, None]).sum(-2)
        S = S + (beta[:, t, :, None] * k[:, t])[..., None] * r[..., None, :]
        o[:, t] = scale * (S * q[:, t, :, :, None]).sum(-2)
    s["state"][at[live]] = S[live]
    return (o * live[:, None, None, None]).to(s["v"].dtype), s["state"]


# ----------------------------------------------------------------------------------- one pass

def run(s):
    if not own:
        if s["op"] == "fwd":
            return _plain_fwd(s)
        if s["op"] == "step":
            return _plain_step(s)
        if s["op"] == "bwd":
            return _plain_bwd(s, s["q"], s["k"], s["v"])
        if s["op"] == "bwd8":
            return _plain_bwd(s, *(_unpack(*s[n], s["d_o"].dtype) for n in ("q", "k", "v")))
        return _unpack(*_pack(s["x"]), s["x"].dtype)
    import chunked_kimi_delta_amd as kda
    if s["op"] == "ckpt":
        return kda.unpack8(kda.pack8(s["x"]))
    raw = dict(use_qk_l2norm=s["raw"], use_beta_sigmoid=s["raw"],
               gate="softplus" if s["gate"] else None, A_log=s["A_log"], dt_bias=s["dt_bias"])
    if s["op"] == "fwd":
        return kda.gdn_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], cu_seqlens=s["cu"],
                           initial_state=s["h0"], **raw)
    if s["op"] == "step":
        o = kda.gdn_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"],
                         state_indices=s["slots"], **raw)
        return o, s["state"]
    q, k, v = s["q"], s["k"], s["v"]
    if s["op"] == "bwd8":
        q, k, v = (kda.Packed8(*x, s["d_o"].dtype) for x in (q, k, v))
    grads = kda.gdn_bwd(q, k, v, s["g"], s["beta"], s["d_o"], s["dht"], cu_seqlens=s["cu"],
                        initial_state=s["h0"], want_dh0=s["h0"] is not None, **raw)
    names = ("dq", "dk", "dv", "dg", "dbeta") + (() if s["h0"] is None else ("dh0",))
    return dict(zip(names, grads))


# ------------------------------------------------------------------------------------- floors

def work(case):
    e = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "ckpt":  # to 8 bits and back
        rows = case["tokens"] * case["heads"]
        return {"bytes": rows * (case["D"] * (2 * e + 2) + 8), "flops": 4 * rows * case["D"]}
    H, G, K, V = case["H"], case["G"], case["K"], case["V"]
    HV = H * G
    if case["op"] == "step":
        live = case["B"] - case["pad"]
        tokens = case["B"] * case["T"]
        return {"bytes": 8 * live * HV * K * V + e * tokens * (2 * H * K + 2 * HV * V + 2 * HV),
                "flops": 7 * live * case["T"] * HV * K * V}
    lens = _lengths(case)
    tokens, states = sum(lens), len(lens) * HV * K * V * 4
    io = tokens * (2 * H * K + HV * V + 2 * HV)  # q, k, v, g, beta
    if case["op"] == "fwd":
        # per token and value head: S^T k, the write, S^T q and the decay
        return {"bytes": e * (io + tokens * HV * V) + states * (2 if case["h0"] else 1),
                "flops": 7 * tokens * HV * K * V}
    kept = io * e
    if case["op"] == "bwd8":
        rows = tokens * (2 * H + HV)
        kept = tokens * (2 * H * K + HV * V) + 4 * rows + e * tokens * 2 * HV
    # the states again, their gradients, and the products of both with every token's rows
    return {"bytes": kept + e * (io + tokens * HV * V) + states * (3 if case["h0"] else 0),
            "flops": 18 * tokens * HV * K * V}


# ------------------------------------------------------------------------------ in 64 bits

def _sequences(s, *xs):
    """Every sequence's rows, padded with zeros: [N, longest, ...]."""
    if s.get("cu") is None:
        return [x.double() for x in xs]
    cu = s["cu"].tolist()
    out = []
    for x in xs:
        y = torch.zeros(len(cu) - 1, s["longest"], *x.shape[2:], dtype=torch.float64, device=x.device)
        for i in range(len(cu) - 1):
            y[i, :cu[i + 1] - cu[i]] = x[0, cu[i]:cu[i + 1]].double()
        out.append(y)
    return out


def _packed(s, like, x):
    if s.get("cu") is None:
        return x
    cu = s["cu"].tolist()
    return torch.cat([x[i, :cu[i + 1] - cu[i]] for i in range(len(cu) - 1)]).reshape(*like)


def _token(S, q, k, v, a, b):
    """One token of every sequence and head: the decayed state, the residual, the new state."""
    D = a[..., None, None] * S
    r = v - torch.matmul(k[..., None, :], D)[..., 0, :]
    return D, r, D + (b[..., None] * k)[..., :, None] * r[..., None, :]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "ckpt":
        x = s["x"].double()
        m = x.abs().amax(-1, keepdim=True)
        return torch.round(x / m * 127) * m / 127
    if case["op"] == "bwd8":  # the values that the checkpoints stand for, in the type kept
        for n in ("q", "k", "v"):
            s[n] = (s[n][0].double() * s[n][1].double()[..., None]).to(s["d_o"].dtype)
    G, K, scale = case["G"], case["K"], case["K"] ** -0.5
    if case["op"] == "step":
        s["cu"] = None
    q0, k0, v, g, b = _sequences(s, s["q"], s["k"], s["v"], s["g"], s["beta"])
    if s["gate"]:
        g = -s["A_log"].double().exp() * torch.nn.functional.softplus(g + s["dt_bias"].double(), threshold=1e9)
    if s.get("cu") is not None:  # rows past a sequence's end neither decay nor write
        n = s["cu"][1:] - s["cu"][:-1]
        on = (torch.arange(s["longest"], device=g.device) < n[:, None]).double()[..., None]
    else:
        on = torch.ones_like(g[..., :1])
    raw = case["raw"]
    root = lambda x: (x.square().sum(-1, keepdim=True) + 1e-6).sqrt()
    qn, kn = (q0 / root(q0), k0 / root(k0)) if raw else (q0, k0)
    ba = (1 / (1 + torch.exp(-b)) if raw else b) * on
    a = torch.exp(g * on)
    q, k = qn.repeat_interleave(G, 2), kn.repeat_interleave(G, 2)
    N, T, HV, V = v.shape
    if case["op"] == "step":
        at = s["slots"].long()
        live = at >= 0
        S = s["state"].double()[at.clamp_min(0)]
    else:
        S = torch.zeros(N, HV, K, V, dtype=torch.float64, device=v.device) if s["h0"] is None else s["h0"].double()
    if case["op"] in ("fwd", "step"):
        o = torch.zeros_like(v)
        for t in range(T):
            S = _token(S, q[:, t], k[:, t], v[:, t], a[:, t], ba[:, t])[2]
            o[:, t] = scale * torch.matmul(q[:, t, :, None, :], S)[..., 0, :]
        if case["op"] == "step":
            pool = s["state"].double()
            pool[at[live]] = S[live]
            return o * live[:, None, None, None], pool
        return _packed(s, s["v"].shape, o), S
    (d_o,) = _sequences(s, s["d_o"])
    step, starts = 64, []
    for t in range(T):
        if t % step == 0:
            starts.append(S)
        S = _token(S, q[:, t], k[:, t], v[:, t], a[:, t], ba[:, t])[2]
    dS = torch.zeros_like(S) if s["dht"] is None else s["dht"].double()
    dq, dk, dv, da, db = (torch.zeros_like(x) for x in (q, k, v, a, ba))
    for c in reversed(range(len(starts))):
        S, kept = starts[c], []
        for t in range(c * step, min(T, c * step + step)):
            kept.append((S, *_token(S, q[:, t], k[:, t], v[:, t], a[:, t], ba[:, t])))
            S = kept[-1][-1]
        for t in reversed(range(c * step, min(T, c * step + step))):
            S0, D, r, S1 = kept[t - c * step]
            dot = d_o[:, t]
            dq[:, t] = scale * torch.matmul(S1, dot[..., None])[..., 0]
            dS = dS + scale * q[:, t, :, :, None] * dot[..., None, :]
            kd = torch.matmul(k[:, t, :, None, :], dS)[..., 0, :]  # dS^T k
            dr = ba[:, t, :, None] * kd
            db[:, t] = (kd * r).sum(-1)
            dk[:, t] = ba[:, t, :, None] * torch.matmul(dS, r[..., None])[..., 0] - torch.matmul(D, dr[..., None])[..., 0]
            dv[:, t] = dr
            dD = dS - k[:, t, :, :, None] * dr[..., None, :]
            da[:, t] = (dD * S0).sum((-1, -2))
            dS = a[:, t, :, None, None] * dD
    dq, dk = (x.unflatten(2, (-1, G)).sum(3) for x in (dq, dk))
    if raw:
        dq = (dq - qn * (qn * dq).sum(-1, keepdim=True)) / root(q0)
        dk = (dk - kn * (kn * dk).sum(-1, keepdim=True)) / root(k0)
        db = db * ba * (1 - ba)
    out = {"dq": dq, "dk": dk, "dv": dv, "dg": da * a, "dbeta": db}
    out = {n: _packed(s, s["g" if n == "dbeta" else n[1:]].shape, x) for n, x in out.items()}
    return out | ({} if s["h0"] is None else {"dh0": dS})
