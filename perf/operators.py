"""The gated delta rule with one decay per head, as measured: chunked forward
and backward, the single-token step, and the 8-bit activation checkpoints that
the backward can start from.

Per value head, with a d_k x d_v state S (its query/key head is shared by
HV / HK value heads):

    S_t = exp(g_t) (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T
    o_t = scale * S_t^T q_t

Sequences are packed one behind the other; `lens` gives their lengths.  The
8-bit form of a tensor is e4m3 with one power-of-two scale for each 32
channels: the smallest one with which the block's largest magnitude does not
pass 448.
"""
import torch

own = False

D = 128            # d_k = d_v
C = 64             # chunk of the plain form
SCALE = D ** -0.5


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # the 8K prefill of 32 value heads, 16 query/key heads, from a kept state
        {"name": "fwd_8k_h32", "op": "fwd", "lens": "8192", "hk": 16, "hv": 32, "gate32": True, "h0": True, "slots": False},
        # a serving batch of ragged prompts whose states live in a pool
        {"name": "fwd_ragged_pool", "op": "fwd", "lens": "1,700,64,2047,333,4096,65,15,1200,63,900,5,1024,128,31,2500",
         "hk": 8, "hv": 16, "gate32": False, "h0": True, "slots": True},
        # one short prompt on a card's share of the heads: latency
        {"name": "fwd_77_h4", "op": "fwd", "lens": "77", "hk": 2, "hv": 4, "gate32": True, "h0": False, "slots": False},
        # pre-training lengths: four sequences of 16K, every head with its own query and key
        {"name": "fwd_b4_16k_h32", "op": "fwd", "lens": "16384,16384,16384,16384", "hk": 32, "hv": 32, "gate32": False, "h0": False, "slots": False},
        # one request's token: latency
        {"name": "step_1_h32", "op": "step", "n": 1, "hk": 16, "hv": 32, "gate32": True, "pad": 0},
        # an odd batch with padded rows, as a captured batch of fixed size has
        {"name": "step_37_h16_pad3", "op": "step", "n": 37, "hk": 16, "hv": 16, "gate32": False, "pad": 3},
        # the 256-request decode of 32 heads
        {"name": "step_256_h32", "op": "step", "n": 256, "hk": 16, "hv": 32, "gate32": True, "pad": 0},
        # q, k and v of 333 tokens and of 16384 tokens into 8 bits and back
        {"name": "pack_333_h8", "op": "pack", "t": 333, "hk": 4, "hv": 8},
        {"name": "pack_16k_h32", "op": "pack", "t": 16384, "hk": 16, "hv": 32},
        # training: gradients of an 8K sequence, final-state gradient included
        {"name": "bwd_8k_h32", "op": "bwd", "lens": "8192", "hk": 16, "hv": 32, "gate32": True, "h0": True, "dht": True, "eight": False},
        # training on packed documents, an odd number of heads
        {"name": "bwd_ragged_h5", "op": "bwd", "lens": "300,1,64,1500,77,2048,33,640", "hk": 5, "hv": 5, "gate32": False, "h0": False, "dht": False, "eight": False},
        # q, k, v checkpointed in 8 bits, then the gradients from them
        {"name": "bwd8_4k_h16", "op": "bwd", "lens": "4000,96", "hk": 8, "hv": 16, "gate32": True, "h0": True, "dht": False, "eight": True},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "step", "pack", "bwd", "bwd"])
    hk = rng.choice([1, 2, 4, 8, 16])
    hv = hk * rng.choice([1, 1, 2, 4])
    while hv > 32:
        hv //= 2
    gate32 = rng.random() < 0.5
    if op == "step":
        return {"op": op, "n": _log(rng, 1, 256), "hk": hk, "hv": hv, "gate32": gate32, "pad": rng.choice([0, 0, 1, 5])}
    if op == "pack":
        return {"op": op, "t": _log(rng, 1, 16384), "hk": hk, "hv": hv}
    n = _log(rng, 1, 12)
    most = 16384 if op == "fwd" else 4096
    lens = ",".join(str(_log(rng, 1, most // n + 1)) for _ in range(n))
    case = {"op": op, "lens": lens, "hk": hk, "hv": hv, "gate32": gate32, "h0": rng.random() < 0.5}
    if op == "fwd":
        case["slots"] = case["h0"] and rng.random() < 0.5
    else:
        case["dht"] = rng.random() < 0.5
        case["eight"] = rng.random() < 0.5
    return case


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


# ------------------------------------------------------------------ inputs --

def _unit(x):
    return x / torch.linalg.vector_norm(x, dim=-1, keepdim=True)


def _tokens(t, hk, hv, gate32, gen):
    """q, k, v as views of one projection's output [t, (2 hk + hv) D], the gate and the write strength."""
    f = dict(generator=gen, device="cuda", dtype=torch.float32)
    qkv = torch.empty((t, (2 * hk + hv) * D), dtype=torch.bfloat16, device="cuda")
    q, k, v = (x.unflatten(-1, (-1, D)) for x in qkv.split([hk * D, hk * D, hv * D], dim=-1))
    q.copy_(_unit(torch.randn((t, hk, D), **f)))
    k.copy_(_unit(torch.randn((t, hk, D), **f)))
    v.copy_(torch.randn((t, hv, D), **f))
    # the decay of a trained layer's shape: -A softplus(a + dt), A in [1, 16], softplus(dt) in [0.001, 0.1]
    a = 1.0 + 15.0 * torch.rand((hv,), **f)
    dt = torch.exp(torch.rand((hv,), **f) * 4.605 - 6.908)
    bias = dt + torch.log(-torch.expm1(-dt))
    g = -a * torch.nn.functional.softplus(torch.randn((t, hv), **f) + bias)
    beta = torch.sigmoid(torch.randn((t, hv), **f))
    kind = torch.float32 if gate32 else torch.bfloat16
    return q, k, v, g.to(kind), beta.to(kind)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    f = dict(generator=gen, device="cuda", dtype=torch.float32)
    s = {"case": case}
    hk, hv = case["hk"], case["hv"]
    if case["op"] == "pack":
        s["q"], s["k"], s["v"], _, _ = _tokens(case["t"], hk, hv, True, gen)
        return s
    if case["op"] == "step":
        n = case["n"] + case["pad"]
        s["q"], s["k"], s["v"], s["g"], s["beta"] = _tokens(n, hk, hv, case["gate32"], gen)
        s["state"] = torch.randn((case["n"] + 2, hv, D, D), **f) * 0.1
        slots = torch.randperm(case["n"] + 2, generator=gen, device="cuda")[:n].to(torch.int32)
        s["slots"] = torch.cat([slots[: case["n"]], torch.full((case["pad"],), -1, dtype=torch.int32, device="cuda")])
        return s
    lens = _lens(case)
    t = sum(lens)
    s["q"], s["k"], s["v"], s["g"], s["beta"] = _tokens(t, hk, hv, case["gate32"], gen)
    s["lens"] = lens
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    # where each token stands in a [sequence, position] array, for the plain form
    at = torch.arange(t, device="cuda")
    seq = torch.bucketize(at, s["cu"][1:].to(torch.int64), right=True)
    s["seq"], s["pos"] = seq, at - s["cu"].to(torch.int64)[seq]
    n = len(lens)
    s["h0"] = torch.randn((n, hv, D, D), **f) * 0.1 if case["h0"] else None
    if case.get("slots"):
        s["pool"] = torch.randn((n + 3, hv, D, D), **f) * 0.1
        s["slots"] = torch.randperm(n + 3, generator=gen, device="cuda")[:n].to(torch.int32)
    if case["op"] == "bwd":
        s["dO"] = torch.randn((t, hv, D), **f).to(torch.bfloat16)
        s["dhT"] = torch.randn((n, hv, D, D), **f) * 0.1 if case["dht"] else None
    return s


# ------------------------------------------------------------- plain forms --

def _spread(s, x, group=1):
    """[t, h, ...] into [sequence, h * group, chunk, C, ...] in 32 bits, zeros behind each sequence."""
    n, most = len(s["lens"]), max(s["lens"])
    chunks = -(-most // C)
    y = x.float()
    y = torch.zeros((n, chunks * C) + x.shape[1:], dtype=torch.float32, device=x.device).index_put((s["seq"], s["pos"]), y)
    y = y.transpose(1, 2).unflatten(2, (chunks, C))
    return y.repeat_interleave(group, dim=1) if group > 1 else y


def _gather(s, y):
    """The packed tokens [t, h, ...] of [sequence, h, chunk, C, ...]."""
    return y.flatten(2, 3).transpose(1, 2)[s["seq"], s["pos"]]


def _plain_chunks(s, q, k, v, g, beta, h0):
    """o [t, hv, D] and the last states, both in 32 bits: chunks of C tokens, inside a chunk
    u = (I + A)^-1 beta (v - decay (k S)) with A the decayed, strictly lower beta k k^T."""
    group = s["case"]["hv"] // s["case"]["hk"]
    q, k, v, g, beta = _spread(s, q, group), _spread(s, k, group), _spread(s, v), _spread(s, g), _spread(s, beta)
    n, hv, chunks = v.shape[:3]
    total = g.double().cumsum(-1)                       # sums of the log-decay, and their differences, in 64 bits
    low = torch.ones((C, C), dtype=torch.bool, device=v.device).tril()
    decay = torch.where(low, total[..., :, None] - total[..., None, :], -torch.inf).exp().float()
    start, end, last = total.exp().float()[..., None], (total[..., -1:] - total).exp().float()[..., None], total[..., -1].exp().float()
    kk = beta[..., None] * (k @ k.transpose(-1, -2)) * decay
    A = torch.where(low & ~torch.eye(C, dtype=torch.bool, device=v.device), kk, 0.0)
    eye = torch.eye(C, device=v.device)
    with torch.no_grad():                               # forward substitution, row by row, all chunks at once
        inv = eye.expand(A.shape).clone()
        for r in range(1, C):
            inv[..., r, :r] = -(A[..., r, None, :r] @ inv[..., :r, :r])[..., 0, :]
    inv = inv @ (2 * eye - (eye + A) @ inv)             # the same values; their derivative is the inverse's
    P = (q @ k.transpose(-1, -2)) * decay
    S = torch.zeros((n, hv, D, D), dtype=torch.float32, device=v.device) if h0 is None else h0
    out = []
    for c in range(chunks):
        u = inv[:, :, c] @ (beta[:, :, c, :, None] * (v[:, :, c] - start[:, :, c] * (k[:, :, c] @ S)))
        out.append(start[:, :, c] * (q[:, :, c] @ S) + P[:, :, c] @ u)
        S = last[:, :, c, None, None] * S + k[:, :, c].transpose(-1, -2) @ (end[:, :, c] * u)
    return _gather(s, torch.stack(out, 2)) * SCALE, S


def _plain_fwd(s):
    h0 = s["h0"]
    if s["case"]["slots"]:
        h0 = s["pool"][s["slots"].long()]
    o, S = _plain_chunks(s, s["q"], s["k"], s["v"], s["g"], s["beta"], h0)
    if s["case"]["slots"]:
        s["pool"].index_copy_(0, s["slots"].long(), S)
        S = s["pool"]
    return {"o": o.to(torch.bfloat16), "state": S}


def _plain_step(s):
    real = s["slots"] >= 0
    at = s["slots"][real].long()
    group = s["case"]["hv"] // s["case"]["hk"]
    q, k, v = (s[x][real].float() for x in "qkv")
    q, k = q.repeat_interleave(group, 1), k.repeat_interleave(group, 1)
    S = s["state"][at] * s["g"][real].float().exp()[..., None, None]
    u = s["beta"][real].float()[..., None] * (v - (k[..., None, :] @ S)[..., 0, :])
    S = S + k[..., :, None] * u[..., None, :]
    o = torch.zeros(s["v"].shape, dtype=torch.bfloat16, device=v.device)
    o[real] = ((q[..., None, :] @ S)[..., 0, :] * SCALE).to(torch.bfloat16)
    s["state"].index_copy_(0, at, S)
    return {"o": o, "state": s["state"]}


def _pow2(e):
    """2^e in 64 bits, exactly (a power function need not be)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _plain_eight(x):
    """The values that the 8-bit form of x stands for, in 32 bits."""
    y = x.float().unflatten(-1, (-1, 32))
    m, e = torch.frexp(y.abs().amax(-1, keepdim=True))
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-127)
    return ((y * _pow2(-e)).float().to(torch.float8_e4m3fn).double() * _pow2(e)).float().flatten(-2)


def _plain_bwd(s):
    leaves = {x: s[x].float() for x in ("q", "k", "v", "g", "beta")}
    if s["case"]["eight"]:
        leaves.update({x: _plain_eight(s[x]) for x in "qkv"})
    if s["h0"] is not None:
        leaves["h0"] = s["h0"].clone()
    for x in leaves.values():
        x.requires_grad_(True)
    o, S = _plain_chunks(s, *(leaves[x] for x in ("q", "k", "v", "g", "beta")), leaves.get("h0"))
    outs, grads = [o], [s["dO"].float()]
    if s["dhT"] is not None:
        outs.append(S)
        grads.append(s["dhT"])
    got = torch.autograd.grad(outs, list(leaves.values()), grads)
    return {"d" + n: x if n == "h0" else x.to(torch.bfloat16) for n, x in zip(leaves, got)}


# -------------------------------------------------------------------- calls --

def run(state):
    s, op = state, state["case"]["op"]
    if own:
        import linear_attention_07_b200 as kda
        if op == "step":
            o = kda.gdn_decode_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], scale=SCALE, slots=s["slots"])
            return {"o": o, "state": s["state"]}
        if op == "pack":
            return dict(zip("qkv", (kda.act_unpack8(x) for x in kda.act_pack8(s["q"], s["k"], s["v"]))))
        q, k, v, g, beta = (s[x].unsqueeze(0) for x in ("q", "k", "v", "g", "beta"))
        if op == "fwd":
            if s["case"]["slots"]:
                o, S = kda.gdn_chunk_fwd(q, k, v, g, beta, s["pool"], scale=SCALE, cu_seqlens=s["cu"], slots=s["slots"])
            else:
                o, S = kda.gdn_chunk_fwd(q, k, v, g, beta, s["h0"], scale=SCALE, cu_seqlens=s["cu"])
            return {"o": o[0], "state": S}
        if s["case"]["eight"]:
            q, k, v = kda.act_pack8(q, k, v)
        got = kda.gdn_chunk_bwd(q, k, v, g, beta, s["h0"], s["dO"].unsqueeze(0), s["dhT"], scale=SCALE, cu_seqlens=s["cu"],
                                want_dh0=s["h0"] is not None)
        out = {n: x[0] for n, x in zip(("dq", "dk", "dv", "dg", "dbeta"), got)}
        if s["h0"] is not None:
            out["dh0"] = got[5]
        return out
    if op == "step":
        return _plain_step(s)
    if op == "pack":
        return {x: _plain_eight(s[x]).to(torch.bfloat16) for x in "qkv"}
    return _plain_fwd(s) if op == "fwd" else _plain_bwd(s)


def work(case):
    hk, hv = case["hk"], case["hv"]
    gate = 4 if case.get("gate32") else 2
    if case["op"] == "pack":
        # each value read once in 16 bits; the 8-bit form written and read; the values written in 16 bits
        return {"bytes": case["t"] * (2 * hk + hv) * D * (2 + 2 * (1 + 1 / 32) + 2), "flops": 0}
    t = case["n"] if case["op"] == "step" else sum(_lens(case))
    n = case["n"] if case["op"] == "step" else len(_lens(case))
    qkv, gates, state = (2 * hk + hv) * D * 2, 2 * hv * gate, hv * D * D * 4
    if case["op"] == "step":
        return {"bytes": t * (qkv + gates + hv * D * 2 + 2 * state), "flops": t * hv * 7 * D * D}
    if case["op"] == "fwd":
        # recall, write and read of the state: three products of d_k x d_v a token
        return {"bytes": t * (qkv + gates + hv * D * 2) + n * state * (2 if case["h0"] else 1), "flops": t * hv * 6 * D * D}
    # the backward: the recall and the write again, and the gradients of the three products
    back = 2 * (2 * hk + hv + hv) * D + 2 * 2 * hv
    moved = t * (qkv + gates + hv * D * 2 + back) + n * state * (2 * case["h0"] + case["dht"])
    if case["eight"]:
        moved += t * (2 * hk + hv) * D * 2 * (1 + 1 / 32)
    return {"bytes": moved, "flops": t * hv * (4 + 12) * D * D}


# ------------------------------------------------------------------- exact --

def _exact_eight(x):
    y = x.double().unflatten(-1, (-1, 32))
    top = y.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(torch.where(top > 0, top, 1.0) / 448))
    e = torch.where(top > 448 * _pow2(e), e + 1, torch.where(top <= 224 * _pow2(e), e - 1, e)).clamp(min=-127)
    z = y / _pow2(e)
    _, bits = torch.frexp(z.abs().clamp(min=2.0 ** -6))    # |z| in [2^(bits - 1), 2^bits): 3 bits behind the leading one
    step = _pow2(bits - 4)
    return (torch.round(z / step) * step * _pow2(e)).flatten(-2)


def _padded(s, x):
    n, most = len(s["lens"]), max(s["lens"])
    y = torch.zeros((most, n) + x.shape[1:], dtype=torch.float64, device=x.device)
    y[s["pos"], s["seq"]] = x.double()
    return y


def _exact_inputs(s, eight):
    group = s["case"]["hv"] // s["case"]["hk"]
    q, k, v = ((_exact_eight(s[x]) if eight else s[x].double()) for x in "qkv")
    q, k = q.repeat_interleave(group, 1), k.repeat_interleave(group, 1)
    return tuple(_padded(s, x) for x in (q * SCALE, k, v, s["g"], s["beta"]))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "pack":
        return {x: _exact_eight(s[x]) for x in "qkv"}
    if case["op"] == "step":
        real = (s["slots"] >= 0).nonzero()[:, 0]
        at = s["slots"][real].long()
        group = case["hv"] // case["hk"]
        q, k, v = (s[x][real].double() for x in "qkv")
        q, k = q.repeat_interleave(group, 1), k.repeat_interleave(group, 1)
        state, o = s["state"].double(), torch.zeros(s["v"].shape, dtype=torch.float64, device="cuda")
        S = torch.exp(s["g"][real].double())[..., None, None] * state[at]
        u = s["beta"][real].double()[..., None] * (v - torch.einsum("nhij,nhi->nhj", S, k))
        S = S + torch.einsum("nhi,nhj->nhij", k, u)
        o[real] = SCALE * torch.einsum("nhij,nhi->nhj", S, q)
        state[at] = S
        return {"o": o, "state": state}
    if case["op"] == "fwd":
        # token by token
        q, k, v, g, beta = _exact_inputs(s, False)
        h0 = s["pool"][s["slots"].long()] if case["slots"] else s["h0"]
        n, hv = v.shape[1:3]
        S = torch.zeros((n, hv, D, D), dtype=torch.float64, device="cuda") if h0 is None else h0.double()
        o = torch.zeros_like(v)
        decay = g.exp()
        for t in range(v.shape[0]):
            S = S * decay[t, ..., None, None]
            u = beta[t, ..., None] * (v[t] - (k[t].unsqueeze(-2) @ S).squeeze(-2))
            S = S + k[t].unsqueeze(-1) * u.unsqueeze(-2)
            o[t] = (q[t].unsqueeze(-2) @ S).squeeze(-2)
        if case["slots"]:
            pool = s["pool"].double()
            pool[s["slots"].long()] = S
            S = pool
        return {"o": o[s["pos"], s["seq"]], "state": S}
    # the backward, token by token: states kept at every 64th token, the tokens between run again
    q, k, v, g, beta = _exact_inputs(s, case["eight"])
    do = _padded(s, s["dO"])
    most, n, hv = v.shape[:3]
    zero = torch.zeros((n, hv, D, D), dtype=torch.float64, device="cuda")
    decay = g.exp()

    def step(S, t):
        """The decayed state, the written value's difference, and the state after token t."""
        Sd = S * decay[t, ..., None, None]
        d = v[t] - (k[t].unsqueeze(-2) @ Sd).squeeze(-2)
        return Sd, d, Sd + k[t].unsqueeze(-1) * (beta[t, ..., None] * d).unsqueeze(-2)

    S = zero if s["h0"] is None else s["h0"].double()
    kept = []
    for t in range(most):
        if t % 64 == 0:
            kept.append(S)
        S = step(S, t)[2]
    dS = zero if s["dhT"] is None else s["dhT"].double()
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, dbeta = torch.zeros_like(g), torch.zeros_like(beta)
    for seg in range(len(kept) - 1, -1, -1):
        S, tape = kept[seg], []
        for t in range(64 * seg, min(most, 64 * seg + 64)):
            tape.append((t,) + step(S, t))
            S = tape[-1][3]
        for t, Sd, d, S1 in reversed(tape):
            dq[t] = (S1 @ do[t].unsqueeze(-1)).squeeze(-1)
            dS = dS + q[t].unsqueeze(-1) * do[t].unsqueeze(-2)
            du = (k[t].unsqueeze(-2) @ dS).squeeze(-2)              # of u = beta d
            dbeta[t] = (du * d).sum(-1)
            dd = beta[t, ..., None] * du
            dv[t] = dd
            dk[t] = (dS @ (beta[t, ..., None] * d).unsqueeze(-1)).squeeze(-1) - (Sd @ dd.unsqueeze(-1)).squeeze(-1)
            dS = dS - k[t].unsqueeze(-1) * dd.unsqueeze(-2)         # of the decayed state
            dg[t] = (dS * Sd).sum((-1, -2))
            dS = dS * decay[t, ..., None, None]
    back = {"dq": dq * SCALE, "dk": dk, "dv": dv, "dg": dg, "dbeta": dbeta}
    out = {x: y[s["pos"], s["seq"]] for x, y in back.items()}
    if case["hv"] != case["hk"]:
        out.update({x: out[x].unflatten(1, (case["hk"], -1)).sum(2) for x in ("dq", "dk")})
    if s["h0"] is not None:
        out["dh0"] = dS
    return out
