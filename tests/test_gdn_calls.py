"""How the calls of the gated delta rule with one decay per head are made:
waits that run out, two calls at once, rows named twice, offsets past 32 bits.

A wait that runs out (KDA_WAIT_LIMIT_NS=0 makes every wait a single check)
faults nothing: the kernels end by themselves, everything that they write is
NaN, kda_device_status says KDA_ERR_TIMEOUT once, and the next call is right.
Tolerances are those of the forward's and the backward's own tests.
"""
import pytest
import torch

import linear_attention_07_b200 as kda
from test_gdn import D, TOL_O, TOL_S, TOL_STEP, batch, cu_of, on_gpu, reference, rel, tokens
from test_gdn_backward import TOL_DG, TOL_GRAD, check, cotangents, run
from test_gdn_backward import reference as gradients

pytestmark = pytest.mark.gpu

LENS = (100, 1, 64)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from linear_attention_07_b200 import build
    build.build()
    kda.load_library()
    torch.cuda.init()


def expired():
    torch.cuda.synchronize()
    assert kda.device_status() == kda.KDA_ERR_TIMEOUT
    assert kda.device_status() == kda.KDA_OK             # read and cleared


def test_forward_waits_expire(monkeypatch):
    x, h0 = tokens(165, 2, 4, seed=70), torch.randn(3, 4, D, D)
    call = lambda: kda.gdn_chunk_fwd(*batch(on_gpu(x)), h0.cuda(), cu_seqlens=cu_of(LENS).cuda())
    assert kda.device_status() == kda.KDA_OK
    monkeypatch.setenv("KDA_WAIT_LIMIT_NS", "0")
    o, S = call()
    expired()
    assert torch.isnan(o.float()).all() and torch.isnan(S).all()
    monkeypatch.delenv("KDA_WAIT_LIMIT_NS")
    o, S = call()
    ro, rS = reference(x, LENS, h0)
    assert rel(o[0], ro) <= TOL_O and rel(S, rS) <= TOL_S
    assert kda.device_status() == kda.KDA_OK


@pytest.mark.parametrize("eight", [False, True])
def test_backward_waits_expire(monkeypatch, eight):
    x, h0 = tokens(165, 2, 4, seed=71), torch.randn(3, 4, D, D)
    dO, dhT = cotangents(165, 4, 3)
    assert kda.device_status() == kda.KDA_OK
    monkeypatch.setenv("KDA_WAIT_LIMIT_NS", "0")
    if eight:
        q, k, v, g, b = batch(on_gpu(x))
        got = kda.gdn_chunk_bwd(*kda.act_pack8(q, k, v), g, b, h0.cuda(), dO[None].cuda(), dhT.cuda(),
                                cu_seqlens=cu_of(LENS).cuda())
    else:
        got = run(x, LENS, dO, h0, dhT)
    expired()
    for name, t in zip(("dq", "dk", "dv", "dg", "dbeta", "dh0"), got):
        assert torch.isnan(t.float()).all(), name
    monkeypatch.delenv("KDA_WAIT_LIMIT_NS")
    check(run(x, LENS, dO, h0, dhT), gradients(x, LENS, dO, h0, dhT))


@pytest.mark.parametrize("lens, heads", [((2600,), (16, 32)), ((5000,), (3, 3)), ((11000, 0, 1, 130), (2, 4)),
                                         ((8300,), (1, 2))], ids=str)
@pytest.mark.parametrize("decay", ["trained", "none"])
def test_long_sequences_of_few_heads(lens, heads, decay):
    """Sequences cut into segments that run at the same time, two or more per sequence."""
    T, N = sum(lens), len(lens)
    x, h0 = tokens(T, *heads, seed=82, decay=decay, beta=0.05 if decay == "none" else None), torch.randn(N, heads[1], D, D)
    n0 = kda.launch_count()
    S = h0.cuda()
    o, _ = kda.gdn_chunk_fwd(*batch(on_gpu(x)), S, cu_seqlens=cu_of(lens).cuda(), hT=S, scale=D ** -0.5)
    assert kda.launch_count() - n0 == 4                  # chunks, first segments, their states joined, the others
    ro, rS = reference(x, lens, h0, scale=D ** -0.5)
    # the start states add the rounding of a transition and of the product with it to the chunks' own
    assert rel(o[0], ro) <= TOL_O and rel(S, rS) <= 2 * TOL_S
    assert kda.device_status() == kda.KDA_OK


@pytest.mark.parametrize("lens, heads", [((2600,), (16, 32)), ((2500,), (5, 5)), ((4500, 0, 1, 130, 6000), (2, 4)), ((5000,), (1, 1))],
                         ids=str)
@pytest.mark.parametrize("ends", [False, True])
def test_gradients_of_long_sequences_of_few_heads(lens, heads, ends):
    """Both chains in segments (32 heads: the forward chain in two parts)."""
    T, N = sum(lens), len(lens)
    x = tokens(T, *heads, seed=86)
    h0 = torch.randn(N, heads[1], D, D) if ends else None
    dO, dhT = cotangents(T, heads[1], N)
    dhT = dhT if ends else None
    n0 = kda.launch_count()
    got = run(x, lens, dO, h0, dhT)
    assert kda.launch_count() - n0 == 6                  # outside, chunks, two of the chains, joined, local
    want = gradients(x, lens, dO, h0, dhT)
    # the start states add the rounding of a transition and of the product with it to the chunks' own
    check(got, want, (TOL_GRAD, TOL_GRAD, TOL_GRAD, TOL_DG, TOL_GRAD, 2 * TOL_S))
    for a, b in zip(got, run(x, lens, dO, h0, dhT)):
        assert torch.equal(a, b)


def test_segments_of_a_batch():
    """Sequences of equal lengths, without cu_seqlens."""
    B, T, HK, HV = 2, 2600, 4, 8
    x, h0 = tokens(B * T, HK, HV, seed=88), torch.randn(B, HV, D, D)
    dO, dhT = cotangents(B * T, HV, B)
    split = [t.unflatten(0, (B, T)) for t in on_gpu(x)]
    n0 = kda.launch_count()
    o, S = kda.gdn_chunk_fwd(*split, h0.cuda())
    assert kda.launch_count() - n0 == 4
    ro, rS = reference(x, [T] * B, h0)
    assert rel(o.flatten(0, 1), ro) <= TOL_O and rel(S, rS) <= 2 * TOL_S
    n0 = kda.launch_count()
    got = kda.gdn_chunk_bwd(*split, h0.cuda(), dO.unflatten(0, (B, T)).cuda(), dhT.cuda())
    assert kda.launch_count() - n0 == 5
    check([t.flatten(0, 1)[None] for t in got[:5]] + [got[5]], gradients(x, [T] * B, dO, h0, dhT),
          (TOL_GRAD, TOL_GRAD, TOL_GRAD, TOL_DG, TOL_GRAD, 2 * TOL_S))


def test_gradients_in_segments_expired(monkeypatch):
    x = tokens(4100, 2, 4, seed=87)
    dO, dhT = cotangents(4100, 4, 1)
    monkeypatch.setenv("KDA_WAIT_LIMIT_NS", "0")
    got = run(x, [4100], dO, None, dhT)
    expired()
    for name, t in zip(("dq", "dk", "dv", "dg", "dbeta", "dh0"), got):
        assert torch.isnan(t.float()).all(), name


@pytest.mark.parametrize("lens, heads", [((30, 9000, 1, 4000), (2, 4)), ((5200, 0, 40, 5300), (1, 2))], ids=str)
def test_long_sequences_in_a_ragged_batch(lens, heads):
    """The long ones go in segments, the others in one piece; a pool in another order, with a row missing."""
    T, N = sum(lens), len(lens)
    x, pool = tokens(T, *heads, seed=84), torch.randn(N + 2, heads[1], D, D)
    slots = torch.randperm(N + 2, generator=torch.Generator().manual_seed(85))[:N].int()
    slots[2] = -1
    kept = [n for n in range(N) if n != 2]
    h0 = torch.where((slots >= 0)[:, None, None, None], pool[slots.long()], 0.0)
    n0 = kda.launch_count()
    S = pool.cuda()
    o, _ = kda.gdn_chunk_fwd(*batch(on_gpu(x)), S, cu_seqlens=cu_of(lens).cuda(), slots=slots.cuda())
    assert kda.launch_count() - n0 == 4
    ro, rS = reference(x, lens, h0)
    assert rel(o[0], ro) <= TOL_O and rel(S[slots.long()[kept]], rS[kept]) <= 2 * TOL_S
    rest = [r for r in range(N + 2) if r not in slots.tolist()]
    assert torch.equal(S[rest].cpu(), pool[rest])
    assert kda.device_status() == kda.KDA_OK


def test_segments_in_a_pool_and_expired(monkeypatch):
    T, HK, HV = 4100, 2, 4
    x, pool = tokens(T, HK, HV, seed=83), torch.randn(3, HV, D, D)
    ro, rS = reference(x, [T], pool[2:])
    for slot in (2, 3):
        S = pool.cuda()
        o, _ = kda.gdn_chunk_fwd(*batch(on_gpu(x)), S, cu_seqlens=cu_of([T]).cuda(), slots=torch.tensor([slot], dtype=torch.int32).cuda())
        if slot == 2:
            assert rel(o[0], ro) <= TOL_O and rel(S[2:], rS) <= 2 * TOL_S
        assert torch.equal(S[:slot].cpu(), pool[:slot])
    assert rel(o[0], reference(x, [T])[0]) <= TOL_O
    monkeypatch.setenv("KDA_WAIT_LIMIT_NS", "0")
    o, S = kda.gdn_chunk_fwd(*batch(on_gpu(x)))
    expired()
    assert torch.isnan(o.float()).all() and torch.isnan(S).all()


def test_two_calls_at_once():
    """Each call has its own workspace: calls on two streams leave one another's results alone."""
    a, b = tokens(1500, 2, 4, seed=72), tokens(1500, 2, 4, seed=73)
    dO, dhT = cotangents(1500, 4, 1)
    xs = [batch(on_gpu(t)) for t in (a, b)]
    dOg, dhTg = dO[None].cuda(), dhT.cuda()

    def both(x):
        o, S = kda.gdn_chunk_fwd(*x)
        return [o, S, *kda.gdn_chunk_bwd(*x, None, dOg, dhTg)]

    want = [both(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[], []]
    for _ in range(4):
        for i, (x, s) in enumerate(zip(xs, streams)):
            with torch.cuda.stream(s):
                got[i].append(both(x))
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        for r in runs:
            assert all(torch.equal(y, z) for y, z in zip(w, r))
    assert kda.device_status() == kda.KDA_OK


def test_two_graphs_of_calls():
    """Captured calls own their workspace too: two graphs replayed in turn and at once."""
    xs = [batch(on_gpu(tokens(700, 2, 2, seed=s))) for s in (74, 75)]
    want = [kda.gdn_chunk_fwd(*x) for x in xs]
    graphs, outs = [], []
    for x in xs:
        s = torch.cuda.Stream()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(kda.gdn_chunk_fwd(*x))
        graphs.append(g)
    for at_once in (False, True):
        for o, S in outs:
            o.zero_()
            S.zero_()
        torch.cuda.synchronize()
        for g in graphs:
            with torch.cuda.stream(torch.cuda.Stream() if at_once else torch.cuda.current_stream()):
                g.replay()
        torch.cuda.synchronize()
        for w, r in zip(want, outs):
            assert all(torch.equal(y, z) for y, z in zip(w, r))


def test_segments_in_a_graph():
    """Calls in segments, captured and replayed with other inputs in the same places."""
    x, y = (batch(on_gpu(tokens(4100, 2, 4, seed=s))) for s in (89, 90))
    dO, dhT = (t.cuda() for t in cotangents(4100, 4, 1))
    dO = dO[None]

    def both(z):
        o, S = kda.gdn_chunk_fwd(*z)
        return [o, S, *kda.gdn_chunk_bwd(*z, None, dO, dhT)]

    want = [both(z) for z in (x, y)]
    held = [t.clone() for t in x]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = both(held)
    for z, w in ((y, want[1]), (x, want[0]), (x, want[0])):
        for a, b in zip(held, z):
            a.copy_(b)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, w))
    assert kda.device_status() == kda.KDA_OK


def test_state_in_place_and_on_a_side_stream():
    x, h0 = tokens(130, 2, 6, seed=76), torch.randn(1, 6, D, D)
    ro, rS = reference(x, [130], h0)
    S = h0.cuda()
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        o, out = kda.gdn_chunk_fwd(*batch(on_gpu(x)), S, hT=S)
        torch.cuda.current_stream().synchronize()
    assert out is S
    assert rel(o[0], ro) <= TOL_O and rel(S, rS) <= TOL_S


def test_a_row_named_twice():
    """Which of two requests a shared row's last state is from is not specified; nothing else is touched."""
    N, HK, HV = 4, 2, 4
    x = tokens(N, HK, HV, seed=77)
    pool = torch.randn(6, HV, D, D)
    slots = torch.tensor([1, 1, 4, 7], dtype=torch.int32)
    S = pool.cuda()
    o = kda.gdn_decode_step(*on_gpu(x), S, slots=slots.cuda())
    assert torch.isfinite(S).all() and torch.isfinite(o.float()).all()
    assert torch.equal(S[[0, 2, 3, 5]].cpu(), pool[[0, 2, 3, 5]])
    assert not o[3].any()
    ro, rS = reference([t[2:3] for t in x], [1], pool[4:5])
    assert rel(o[2], ro[0]) <= TOL_O and rel(S[4:5], rS) <= TOL_STEP
    S = pool.cuda()
    kda.gdn_chunk_fwd(*batch(on_gpu(x)), S, cu_seqlens=cu_of([1] * N).cuda(), slots=slots.cuda())
    assert torch.isfinite(S).all()
    assert torch.equal(S[[0, 2, 3, 5]].cpu(), pool[[0, 2, 3, 5]])
    assert rel(S[4:5], rS) <= TOL_S
    assert kda.device_status() == kda.KDA_OK


def test_pool_past_32_bits():
    """Rows behind the 2^31st element of a pool."""
    HK, HV, rows = 2, 32, 4099
    assert (rows - 1) * HV * D * D > 2 ** 31
    pool = torch.empty(rows, HV, D, D, device="cuda")
    S0 = torch.randn(2, HV, D, D)
    rws = torch.tensor([rows - 1, rows - 3])
    pool[rws] = S0.cuda()
    slots = rws.int().cuda()
    x = tokens(2, HK, HV, seed=78)
    o = kda.gdn_decode_step(*on_gpu(x), pool, slots=slots)
    ro, rS = reference(x, [1, 1], S0)
    assert rel(o, ro) <= TOL_O and rel(pool[rws], rS) <= TOL_STEP
    pool[rws] = S0.cuda()
    x = tokens(80, HK, HV, seed=79)
    o, _ = kda.gdn_chunk_fwd(*batch(on_gpu(x)), pool, cu_seqlens=cu_of([70, 10]).cuda(), slots=slots)
    ro, rS = reference(x, [70, 10], S0)
    assert rel(o[0], ro) <= TOL_O and rel(pool[rws], rS) <= TOL_S


def test_tokens_past_32_bits():
    """A sequence whose values lie behind the 2^31st element of v and o."""
    HK, HV, L = 1, 64, 100
    T = 2 ** 31 // (HV * D) + 200
    x = tokens(L, HK, HV, seed=80)
    big = []
    for t in x:
        y = torch.zeros(1, T, *t.shape[1:], dtype=t.dtype, device="cuda")
        y[0, T - L:] = t.cuda()
        big.append(y)
    cu = torch.tensor([T - L - 30, T - L, T], dtype=torch.int32, device="cuda")
    o, S = kda.gdn_chunk_fwd(*big, cu_seqlens=cu)
    ro, rS = reference(x, [L])
    assert rel(o[0, T - L:], ro) <= TOL_O and rel(S[1:], rS) <= TOL_S
    del o
    back = kda.act_unpack8(kda.act_pack8(big[2]))
    small = kda.act_unpack8(kda.act_pack8(x[2].cuda().contiguous()))
    assert torch.equal(back[0, T - L:], small) and not back[0, :T - L].any()


def test_strides_past_32_bits():
    """Tokens so far apart that the last ones lie behind the 2^31st element of their tensor."""
    HK, HV, T = 2, 4, 130
    x = tokens(T, HK, HV, seed=81)
    dO, dhT = cotangents(T, HV, 1)
    stride = 2 ** 24 + 2 ** 19
    assert (T - 1) * stride > 2 ** 31
    wide = torch.empty(1, T, stride, dtype=torch.bfloat16, device="cuda")
    far, at = [], stride - (2 * HK + HV) * D
    for t in x[:3]:
        heads = t.shape[1]
        y = wide[..., at:at + heads * D].unflatten(-1, (heads, D))
        y.copy_(t[None].cuda())
        far.append(y)
        at += heads * D
    gates = batch([t.cuda() for t in x[3:]])
    near = batch(on_gpu(x))
    for a, b in zip(kda.gdn_chunk_fwd(*far, *gates), kda.gdn_chunk_fwd(*near)):
        assert torch.equal(a, b)
    back = lambda y: kda.gdn_chunk_bwd(*y, *gates, None, dO[None].cuda(), dhT.cuda())
    for a, b in zip(back(far), back(near[:3])):
        assert torch.equal(a, b)
    for a, b in zip(kda.act_pack8(*far), kda.act_pack8(*near[:3])):
        assert torch.equal(a.data.view(torch.uint8), b.data.view(torch.uint8)) and torch.equal(a.scales, b.scales)


def random_offsets(N, T, seed, ordered=False):
    cu = torch.randint(-100, T + 100, (N + 1,), generator=torch.Generator().manual_seed(seed))
    return (cu.sort()[0] if ordered else cu).tolist()


# an empty range in front of one that begins earlier, above and below 32 sequences; long ones in segments; all of nothing
BACK = {"empty before an earlier one": (256, [200, 20, 60]),
        "two in the wrong order": (300, [200, 300, 0, 100]),
        "one end too far": (500, [0, 100, 1 << 30, 200, 400]),
        "random": (700, random_offsets(20, 700, 1)),
        "random, more than 32": (700, random_offsets(70, 700, 2)),
        "one goes back, more than 32": (2000, sorted(range(0, 2000, 50)) + [300, 1950, 2000]),
        "segments": (6000, [0, 2500, 100, 6000]),
        "below zero": (100, [-5, -(1 << 31), -7])}


@pytest.mark.parametrize("name", list(BACK))
def test_offsets_that_go_back(name):
    """An offset counts as the largest up to it, inside the tokens: bit for bit what the offsets written so give, with
    nothing left of the call before, whose workspace this one takes."""
    T, cu = BACK[name]
    N, HK, HV = len(cu) - 1, 1, 2
    kept = torch.tensor(cu).clamp(0, T).cummax(0)[0].int()
    cu = torch.tensor(cu, dtype=torch.int32)
    other, x = (batch(on_gpu(tokens(T, HK, HV, seed=s))) for s in (91, 92))
    h0 = torch.randn(N, HV, D, D, generator=torch.Generator().manual_seed(93)).cuda()
    dO, dhT = cotangents(T, HV, N)
    dO, dhT = dO[None].cuda(), dhT.cuda()

    def both(y, offsets):
        o = torch.full((1, T, HV, D), 7.0, dtype=torch.bfloat16, device="cuda")
        _, S = kda.gdn_chunk_fwd(*y, h0, cu_seqlens=offsets.cuda(), o=o)
        back = kda.gdn_chunk_bwd(*y, h0, dO, dhT, cu_seqlens=offsets.cuda())
        packed = kda.gdn_chunk_bwd(*kda.act_pack8(*y[:3]), *y[3:], h0, dO, dhT, cu_seqlens=offsets.cuda())
        return [o, S, *back, *packed]

    both(other, cu_of([T // N] * N))
    got = both(x, cu)
    both(other, cu_of([T // N] * N))
    for a, b in zip(got, both(x, kept)):
        assert torch.equal(a, b)
    first, last = int(kept[0]), int(kept[-1])
    for t, outside in zip(got[:1] + got[2:7], [7, 0, 0, 0, 0, 0]):
        assert (t[0, :first] == outside).all() and (t[0, last:] == outside).all()
    for n in range(N):
        if kept[n] == kept[n + 1]:
            assert torch.equal(got[1][n], h0[n]) and torch.equal(got[7][n], dhT[n])
    assert kda.device_status() == kda.KDA_OK


def test_many_sequences():
    """More sequences than a warp has lanes, more than its square, empty ones among them."""
    for N, seed in ((33, 1), (130, 2), (1100, 3)):
        lens = torch.randint(0, 5, (N,), generator=torch.Generator().manual_seed(seed)).tolist()
        lens[N // 2] = 150
        T = sum(lens) + 7
        x = tokens(T, 1, 2, seed=94 + seed)
        ro, rS = reference(x, lens, begin=3)
        dO, dhT = cotangents(T, 2, N)
        cu = cu_of(lens, 3).cuda()
        o = torch.zeros(1, T, 2, D, dtype=torch.bfloat16, device="cuda")
        _, S = kda.gdn_chunk_fwd(*batch(on_gpu(x)), cu_seqlens=cu, o=o)
        assert rel(o[0], ro) <= TOL_O and rel(S, rS) <= TOL_S
        check(kda.gdn_chunk_bwd(*batch(on_gpu(x)), None, dO[None].cuda(), dhT.cuda(), cu_seqlens=cu),
              gradients(x, lens, dO, None, dhT, begin=3))


def test_fp32_decay_with_bf16_write_strength():
    """Bit for bit what both in fp32 give, the write strength's values being the same."""
    x, h0 = tokens(300, 2, 4, seed=98), torch.randn(3, 4, D, D, generator=torch.Generator().manual_seed(99)).cuda()
    q, k, v, g, b = batch(on_gpu(x))
    b = b.to(torch.bfloat16)
    cu = cu_of([100, 7, 193]).cuda()
    dO, dhT = cotangents(300, 4, 3)
    dO, dhT = dO[None].cuda(), dhT.cuda()

    def calls(beta):
        S = h0.clone()
        step = kda.gdn_decode_step(*(t[0, :3] for t in (q, k, v, g, beta)), S)
        return [*kda.gdn_chunk_fwd(q, k, v, g, beta, h0, cu_seqlens=cu), step, S,
                *kda.gdn_chunk_bwd(q, k, v, g, beta, h0, dO, dhT, cu_seqlens=cu),
                *kda.gdn_chunk_bwd(*kda.act_pack8(q, k, v), g, beta, h0, dO, dhT, cu_seqlens=cu)]

    for a, w in zip(calls(b), calls(b.float())):
        assert a.dtype == w.dtype and torch.equal(a, w)
    with pytest.raises(TypeError):
        kda.gdn_chunk_fwd(q, k, v, g.to(torch.bfloat16), b.float(), cu_seqlens=cu)
    assert kda.device_status() == kda.KDA_OK


FIRST_CALL = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
import linear_attention_07_b200 as kda
from test_gdn import batch, on_gpu, tokens
from test_gdn_backward import cotangents
x = batch(on_gpu(tokens(2200, 2, 4, seed=100)))
dO, dhT = (t.cuda() for t in cotangents(2200, 4, 1))
S = torch.zeros(1, 4, 128, 128, device="cuda")
def calls():
    o, h = kda.gdn_chunk_fwd(*x)
    packed = kda.act_pack8(*x[:3])
    return [o, h, *kda.gdn_chunk_bwd(*packed, *x[3:], None, dO[None], dhT), kda.gdn_decode_step(*(t[0, :1] for t in x), S)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = calls()
graph.replay()
torch.cuda.synchronize()
S.zero_()
assert all(torch.equal(a, b) for a, b in zip(got, calls()))
assert kda.device_status() == kda.KDA_OK
print("captured first")
"""


def test_first_call_of_a_process_is_captured():
    """What a call sets up once per device may happen inside a capture."""
    import os
    import subprocess
    import sys
    tests = os.path.dirname(os.path.abspath(__file__))
    code = FIRST_CALL.format(root=os.path.dirname(tests), tests=tests)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr


def test_calls_from_threads():
    """Calls from several host threads, each on a stream of its own."""
    import threading
    xs = [batch(on_gpu(tokens(T, 2, 4, seed=101 + T))) for T in (100, 700, 2300)]
    dOs = [cotangents(x[0].shape[1], 4, 1) for x in xs]
    dOs = [(a[None].cuda(), b.cuda()) for a, b in dOs]

    def calls(i):
        x, (dO, dhT) = xs[i], dOs[i]
        o, S = kda.gdn_chunk_fwd(*x)
        packed = kda.act_pack8(*x[:3])
        return [o, S, *kda.gdn_chunk_bwd(*x, None, dO, dhT), *kda.gdn_chunk_bwd(*packed, *x[3:], None, dO, dhT),
                *(kda.act_unpack8(p) for p in packed)]

    want = [calls(i) for i in range(3)]
    torch.cuda.synchronize()
    wrong = []

    def thread(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(6):
                    got = calls(i)
                    torch.cuda.current_stream().synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                        wrong.append(i)
        except Exception as e:
            wrong.append(e)

    threads = [threading.Thread(target=thread, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
    assert kda.device_status() == kda.KDA_OK


NO_MEMORY = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
import linear_attention_07_b200 as kda
T, HK, HV = 16384, 1, 64
q, k = (torch.randn(1, T, HK, 128, device="cuda").to(torch.bfloat16) for _ in range(2))
v = torch.randn(1, T, HV, 128, device="cuda").to(torch.bfloat16)
g, b = -torch.rand(1, T, HV, device="cuda"), torch.rand(1, T, HV, device="cuda")
o, S = torch.empty_like(v), torch.zeros(1, HV, 128, 128, device="cuda")
kda.act_pack8(k)
torch.cuda.empty_cache()
free, _ = torch.cuda.mem_get_info()
held = torch.empty(free - (700 << 20), dtype=torch.uint8, device="cuda")      # of 1.09 GB of workspace
for _ in range(2):
    try:
        kda.gdn_chunk_fwd(q, k, v, g, b, o=o, hT=S)
        raise SystemExit("there was memory")
    except kda.KdaError as e:
        assert e.status == kda.KDA_ERR_NO_MEMORY, e
    assert not S.any()
    kda.act_pack8(k)                    # not blamed for it
    kda.gdn_decode_step(*(t[0, :1] for t in (q, k, v, g, b)), S)
    S.zero_()
del held
torch.cuda.empty_cache()
kda.gdn_chunk_fwd(q, k, v, g, b, o=o, hT=S)
torch.cuda.synchronize()
assert S.any() and kda.device_status() == kda.KDA_OK
print("said so")
"""


def test_no_memory_for_the_workspace():
    """KDA_ERR_NO_MEMORY, nothing written, and the calls behind it go on."""
    import os
    import subprocess
    import sys
    tests = os.path.dirname(os.path.abspath(__file__))
    code = NO_MEMORY.format(root=os.path.dirname(tests), tests=tests)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "said so" in r.stdout, r.stderr
