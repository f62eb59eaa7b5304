"""The gated delta rule with one decay per head (kda_gdn_*): against the fp64
oracle, which takes the decay per channel (the same value in every channel).

Tolerances.  bf16 outputs: rounding to nearest is off by at most 2^-8 of the
value, uniformly spread over that range by 2^-8 / sqrt(3) in the root mean
square.  TOL_O = 2^-8 leaves room for three such roundings (U and P inside a
chunk, o itself) in quadrature; the kernels have the last one only, and what
their pairs of bf16 keep is held in test_gdn_digits.py.  fp32 states: operands
enter as pairs of bf16, off by at most 2^-16; 5 * 2^-16 is five such errors at
once, for every chunk, since a chunk's own error shrinks with the state it is
part of (TOL_S).  The single
step is fp32 throughout: sums of 128 terms, 128 * 2^-24 (TOL_STEP).
"""
import numpy as np
import pytest
import torch

import linear_attention_07_b200 as kda

TOL_O = 2.0 ** -8
TOL_S = 5 * 2.0 ** -16
TOL_STEP = 128 * 2.0 ** -24
D = 128


def rel(x, ref):
    x = x.detach().double().cpu().numpy() if hasattr(x, "detach") else np.asarray(x, np.float64)
    ref = ref.detach().double().cpu().numpy() if hasattr(ref, "detach") else np.asarray(ref, np.float64)
    assert x.shape == ref.shape, (x.shape, ref.shape)
    assert np.isfinite(x).all()
    # fp32 has nothing below 2^-149: a reference whose norm is near that (decays of exp(-100) and less) counts as
    # zero, to 2^-120, 2^29 times the smallest fp32 number
    n = max(float(np.linalg.norm(ref)), 2.0 ** -120)
    return float(np.linalg.norm(x - ref)) / n


def tokens(T, HK, HV, *, seed, dk=D, dv=D, gate=torch.float32, decay="trained", beta=None, repeat=False):
    """q, k, v as slices of one tensor [T, (2 HK + HV) d], gates, on the host."""
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen)
    qkv = torch.zeros(T, 2 * HK * dk + HV * dv, dtype=torch.bfloat16)
    q, k, v = qkv.split([HK * dk, HK * dk, HV * dv], dim=-1)
    q, k, v = q.unflatten(-1, (HK, dk)), k.unflatten(-1, (HK, dk)), v.unflatten(-1, (HV, dv))
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)
    q.copy_(unit(rn(T, HK, dk)))
    k.copy_(unit(rn(1, HK, dk)).expand(T, HK, dk) if repeat else unit(rn(T, HK, dk)))
    v.copy_(rn(T, HV, dv))
    g = {"trained": -torch.exp(rn(T, HV) - 3), "none": torch.zeros(T, HV), "strong": torch.full((T, HV), -5.0),
         "far": -200.0 * torch.rand(T, HV, generator=gen),
         "reset": torch.where(torch.rand(T, HV, generator=gen) < 0.1, -torch.inf, -0.01)}[decay]
    b = torch.sigmoid(rn(T, HV)) if beta is None else torch.full((T, HV), float(beta))
    return q, k, v, g.to(gate), b.to(gate)


def reference(x, lens, h0=None, scale=1.0, begin=0):
    """o [T, HV, dv] (zeros outside the sequences) and the last states [N, HV, dk, dv], fp64."""
    import oracle
    q, k, v, g, b = (t.double() for t in x)
    T, HK, dk = q.shape
    HV, dv = v.shape[1:]
    q, k = (t.repeat_interleave(HV // HK, 1) for t in (q * scale, k))
    gc = g[..., None].expand(T, HV, dk)
    o = np.zeros((T, HV, dv))
    S = np.zeros((len(lens), HV, dk, dv))
    at = begin
    for n, L in enumerate(lens):
        sl = slice(at, at + L)
        h = None if h0 is None else h0[n:n + 1]
        if L:
            on, Sn = oracle.fwd(*(t[None, sl] for t in (q, k, v, gc, b)), h)
            o[sl], S[n] = on[0], Sn[0]
        elif h is not None:
            S[n] = h[0].double().numpy()
        at += L
    return o, S


def cu_of(lens, begin=0):
    return torch.tensor(np.cumsum([begin] + list(lens)), dtype=torch.int32)


def on_gpu(x):
    """The same layout on the GPU: slices of one tensor stay slices."""
    q, k, v, g, b = x
    base = q._base if q._base is not None else None
    d = base.cuda()
    HK, dk = q.shape[1:]
    HV, dv = v.shape[1:]
    qd, kd, vd = d.split([HK * dk, HK * dk, HV * dv], dim=-1)
    return [qd.unflatten(-1, (HK, dk)), kd.unflatten(-1, (HK, dk)), vd.unflatten(-1, (HV, dv)), g.cuda(), b.cuda()]


def batch(x):
    return [t[None] for t in x]


# ---------------------------------------------------------------- refusals --

def _host(**kw):
    x = tokens(4, 2, 4, seed=0)
    return batch(x)


def test_refusals_on_the_host():
    """The C calls refuse bad arguments before any launch."""
    import ctypes
    lib = kda.load_library()
    n0 = lib.kda_launch_count()
    A, B2, MIS, NUL = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x20000), ctypes.c_void_p(0x10008), None
    E, U = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED

    def fwd(q=A, k=A, v=A, g=A, beta=A, h0=NUL, o=A, hT=B2, cu=NUL, slots=NUL, n_slots=0, N=2, T=64, HK=2, HV=4,
            dk=128, dv=128, qs=256, ks=256, vs=512, gf=1):
        return lib.kda_gdn_chunk_fwd(q, k, v, g, beta, h0, o, hT, cu, slots, n_slots, 1.0, N, T, HK, HV, dk, dv, qs, ks,
                                     vs, gf, None)

    for bad in (dict(q=NUL), dict(o=NUL), dict(k=MIS), dict(v=NUL), dict(g=NUL), dict(beta=NUL), dict(h0=MIS),
                dict(hT=MIS), dict(HK=3), dict(HK=0), dict(qs=248), dict(qs=260), dict(vs=504), dict(T=-1), dict(N=-1),
                dict(n_slots=-1), dict(cu=ctypes.c_void_p(0x10002)), dict(slots=ctypes.c_void_p(0x10001)),
                dict(g=ctypes.c_void_p(0x10002)), dict(dk=0)):
        assert fwd(**bad) == E, bad
    for bad in (dict(dk=64, qs=256), dict(dv=64), dict(T=1 << 30, N=4), dict(HK=70000, HV=70000, qs=1 << 24, ks=1 << 24, vs=1 << 24)):
        assert fwd(**bad) == U, bad
    assert fwd(N=0) == kda.KDA_OK and fwd(HK=0, HV=0) == kda.KDA_OK
    assert fwd(T=0, hT=NUL, q=NUL, k=NUL, v=NUL, o=NUL, g=NUL, beta=NUL) == kda.KDA_OK

    def step(q=A, state=A, o=A, slots=NUL, n_slots=0, N=2, HK=2, HV=4, dk=128, dv=128, qs=256, vs=512, g=A):
        return lib.kda_gdn_decode_step(q, A, A, g, A, state, o, slots, n_slots, 1.0, N, HK, HV, dk, dv, qs, 256, vs, 1, None)

    for bad in (dict(q=NUL), dict(state=NUL), dict(state=MIS), dict(o=MIS), dict(HK=3), dict(qs=255), dict(N=-1), dict(g=NUL),
                dict(n_slots=-1)):
        assert step(**bad) == E, bad
    assert step(dk=96, qs=256) == U and step(dv=256, vs=1024) == U
    assert step(N=0, q=NUL) == kda.KDA_OK
    assert lib.kda_launch_count() == n0


def test_refusals_of_the_binding():
    x = _host()
    with pytest.raises(ValueError, match="CUDA"):
        kda.gdn_chunk_fwd(*x)
    with pytest.raises(ValueError, match="CUDA"):
        kda.gdn_decode_step(*[t[0] for t in x], torch.zeros(4, 4, D, D))


def test_gate_types():
    """Both fp32, both bf16, or an fp32 decay with a bf16 write strength."""
    kda._types()
    f, b = torch.zeros(2, 4), torch.zeros(2, 4, dtype=torch.bfloat16)
    of = lambda g, beta: kda._check_gates(g, beta, (2, 4), g.device)[2]
    assert (of(b, b), of(f, f), of(f, b)) == (0, 1, kda.GATE_F32_BETA_BF16)
    for g, beta in ((b, f), (f.double(), f), (f, f.double()), (f.half(), b), (b, b.half()), (f, b.half()), (f.int(), f)):
        with pytest.raises(TypeError):
            of(g, beta)
    for g, beta in ((f, b[:1]), (f[:, ::2], b), (f, b.t())):
        with pytest.raises(ValueError):
            of(g, beta)
    import ctypes
    lib, A = kda.load_library(), ctypes.c_void_p(0x10000)
    n0 = lib.kda_launch_count()
    for gate, g, beta in ((2, 0x10002, 0x10000), (2, 0x10000, 0x10001), (2, 0x10000, 0), (2, 0, 0x10000), (1, 0x10000, 0x10002),
                          (3, 0x10000, 0x10002), (0, 0x10001, 0x10000)):
        P = ctypes.c_void_p
        assert lib.kda_gdn_chunk_fwd(A, A, A, P(g), P(beta), None, A, None, None, None, 0, 1.0, 1, 64, 2, 4, 128, 128, 256, 256,
                                     512, gate, None) == kda.KDA_ERR_INVALID_ARG
        assert lib.kda_gdn_decode_step(A, A, A, P(g), P(beta), A, A, None, 0, 1.0, 1, 2, 4, 128, 128, 256, 256, 512, gate,
                                       None) == kda.KDA_ERR_INVALID_ARG
        assert lib.kda_gdn_chunk_bwd(A, A, A, P(g), P(beta), None, A, None, A, A, A, A, A, A, None, 1.0, 1, 64, 2, 4, 128, 128,
                                     256, 256, 512, gate, None) == kda.KDA_ERR_INVALID_ARG
    assert lib.kda_launch_count() == n0


BROADCAST = [((1, 1, 2, D), (1, 4096, 2, D)), ((1, 2, D), (64, 2, D)), ((1, 1, 2, D), (8, 1, 2, D)),
             ((3, 1, 2, D), (3, 5, 2, D)), ((1, 5, 2, D), (3, 5, 2, D)), ((2, 1, 4, 1, 2, D), (2, 3, 4, 1, 2, D)),
             ((D,), (5, 1, D))]


@pytest.mark.parametrize("shape, wide", BROADCAST, ids=str)
def test_broadcast_tokens_are_refused(shape, wide):
    """A token axis of stride 0 names the same values again: the kernels, which step from token to token, would
    read behind the tensor."""
    kda._types()
    x = torch.zeros(shape, dtype=torch.bfloat16).expand(wide)
    with pytest.raises(ValueError, match="token"):
        kda._check_tokens(x, "q", x.shape[:-2], *x.shape[-2:], x.device)
    y = x.contiguous()
    assert kda._check_tokens(y, "q", y.shape[:-2], *y.shape[-2:], y.device) == y.shape[-2] * D


def test_token_strides():
    """The stride of slices of a wider tensor; axes of one entry do not matter; uneven ones are refused."""
    kda._types()
    wide = torch.zeros(3, 5, 8, D, dtype=torch.bfloat16)
    of = lambda t: kda._check_tokens(t, "q", t.shape[:-2], *t.shape[-2:], t.device)
    assert of(wide[:, :, 2:4]) == 8 * D and of(wide[:1, :, 2:4]) == 8 * D and of(wide[:, :1, :4]) == 5 * 8 * D
    assert of(wide[1:2, 2:3, :4]) == 4 * D and of(wide[:, ::2, :4][:1]) == 16 * D
    assert of(wide[:1, :1, :4].expand(1, 1, 4, D)) == 4 * D
    for bad in (wide[:, :4, :4], wide[:, :, ::2], wide.transpose(0, 1)[..., :4, :], wide[..., :64]):
        with pytest.raises(ValueError):
            of(bad)


# ------------------------------------------------------------ chunked forward --

SHAPES = [(1,), (2, 1), (15,), (16, 17), (63, 64, 65), (127, 0, 128, 129), (0, 5, 0), (200, 1, 1, 333)]


@pytest.mark.gpu
@pytest.mark.parametrize("lens", SHAPES, ids=str)
@pytest.mark.parametrize("h0", [False, True])
def test_forward_ragged(lens, h0):
    """Every length around the chunk's borders, packed; grouped heads; both gate types."""
    HK, HV = 2, 4
    for gate in (torch.float32, torch.bfloat16):
        x = tokens(sum(lens), HK, HV, seed=sum(lens) + 7, gate=gate)
        h = torch.randn(len(lens), HV, D, D, generator=torch.Generator().manual_seed(3)) * 0.1 if h0 else None
        ro, rS = reference(x, lens, h, scale=0.3)
        o, S = kda.gdn_chunk_fwd(*batch(on_gpu(x)), None if h is None else h.cuda(), scale=0.3, cu_seqlens=cu_of(lens).cuda())
        assert rel(o[0], ro) <= TOL_O
        assert rel(S, rS) <= TOL_S
        assert kda.device_status() == kda.KDA_OK


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [(1, 1), (3, 3), (2, 10), (5, 15), (16, 16)], ids=str)
def test_forward_heads_in_a_batch(heads):
    """Equal lengths without cu_seqlens, head counts of all kinds, dense tensors."""
    HK, HV = heads
    B, T = 2, 100
    x = tokens(B * T, HK, HV, seed=HV)
    ro, rS = reference(x, [T] * B)
    y = [t.reshape(B, T, *t.shape[1:]).contiguous().cuda() for t in x]
    o, S = kda.gdn_chunk_fwd(*y)
    assert rel(o.flatten(0, 1), ro) <= TOL_O
    assert rel(S, rS) <= TOL_S


@pytest.mark.gpu
@pytest.mark.parametrize("decay", ["none", "strong", "far", "reset"])
@pytest.mark.parametrize("beta", [None, 0.0, 1.0])
def test_forward_decays(decay, beta):
    """No decay, decays far below any floor, tokens that reset the state (log-decay -inf)."""
    x = tokens(200, 1, 2, seed=11, decay=decay, beta=beta)
    ref = list(x)
    ref[3] = torch.clamp(x[3], min=-1e4)            # exp is zero there in 64 bits as well
    h = torch.randn(1, 2, D, D, generator=torch.Generator().manual_seed(4)) * 0.1
    ro, rS = reference(ref, [200], h)
    o, S = kda.gdn_chunk_fwd(*batch(on_gpu(x)), h.cuda())
    assert rel(o[0], ro) <= TOL_O
    assert rel(S, rS) <= TOL_S


@pytest.mark.gpu
@pytest.mark.parametrize("decay", ["trained", "none", "strong", "far", "reset"])
def test_forward_is_linear_in_the_values(decay):
    """o and hT are linear in (v, h0), however small or large these are: powers of two scale every bit of them. 2^-30 and
    2^30 leave every number that counts (down to 2^-60 of the largest) a normal one, so no rounding changes."""
    lens = [150, 65, 1, 64]
    x = tokens(sum(lens), 2, 4, seed=16, decay=decay)
    ref = list(x)
    ref[3] = torch.clamp(x[3], min=-1e4)
    h = torch.randn(4, 4, D, D, generator=torch.Generator().manual_seed(6))
    for h0 in (None, h):
        results = []
        for e in (0, -30, 30):
            f = 2.0 ** e
            y = on_gpu(x)
            y[2].copy_(y[2] * f)
            o, S = kda.gdn_chunk_fwd(*batch(y), None if h0 is None else (h0 * f).cuda(), cu_seqlens=cu_of(lens).cuda())
            results.append((o.double() / f, S.double() / f))
        ro, rS = reference(ref, lens, h0)
        for o, S in results:
            assert rel(o[0], ro) <= TOL_O and rel(S, rS) <= TOL_S
            for a, b in ((o, results[0][0]), (S, results[0][1])):
                top = b.abs().max()
                counts = b.abs() >= top * 2.0 ** -60
                assert torch.equal(a[counts], b[counts])
                assert bool((a[~counts].abs() <= top * 2.0 ** -59).all())


@pytest.mark.gpu
def test_forward_repeated_keys():
    """The same key at every token: A is dense, and powers of A would lose every digit."""
    x = tokens(256, 1, 2, seed=12, decay="none", beta=0.9, repeat=True)
    ro, rS = reference(x, [256])
    o, S = kda.gdn_chunk_fwd(*batch(on_gpu(x)))
    assert rel(o[0], ro) <= TOL_O
    # the key's norm is 1 up to bf16; the sums of U over 64 equal keys cancel to the last value
    assert rel(S, rS) <= 64 * TOL_S


@pytest.mark.gpu
def test_forward_long():
    x = tokens(5000, 2, 2, seed=13)
    ro, rS = reference(x, [5000])
    o, S = kda.gdn_chunk_fwd(*batch(on_gpu(x)))
    assert rel(o[0], ro) <= TOL_O
    assert rel(S, rS) <= TOL_S


@pytest.mark.gpu
def test_forward_pool_padding_and_untouched_rows():
    """A pool of states with padded sequences; rows of o outside the sequences and rows of the pool that no
    sequence names stay as they were; NaN and infinities in tokens that belong to nobody or to a neighbour
    stay there."""
    lens, begin, T = [70, 0, 33, 64], 5, 200
    x = tokens(T, 2, 4, seed=21)
    for t in x[:3]:
        t[:5] = float("nan")
        t[172:] = float("inf")
    x[3][172:], x[4][:5] = float("nan"), float("nan")
    used = [t[5:172] for t in x]
    pool = torch.randn(9, 4, D, D, generator=torch.Generator().manual_seed(5)) * 0.1
    slots = torch.tensor([7, 2, -1, 0], dtype=torch.int32)
    h = torch.stack([pool[7], pool[2], torch.zeros_like(pool[0]), pool[0]])
    ro, rS = reference(used, lens, h)
    dpool = pool.cuda()
    o = torch.full((1, T, 4, D), 7.0, dtype=torch.bfloat16, device="cuda")
    out, ret = kda.gdn_chunk_fwd(*batch(on_gpu(x)), dpool, cu_seqlens=cu_of(lens, begin).cuda(), slots=slots.cuda(), o=o)
    assert out is o and ret is dpool
    assert rel(o[0, 5:172], ro) <= TOL_O
    assert bool((o[0, :5] == 7).all()) and bool((o[0, 172:] == 7).all())
    got = dpool.cpu()
    for r, n in ((7, 0), (2, 1), (0, 3)):
        assert rel(got[r], rS[n]) <= TOL_S
    for r in (1, 3, 4, 5, 6, 8):
        assert torch.equal(got[r], pool[r])
    # a slot past the pool is a padded sequence too
    before = dpool.clone()
    o2, _ = kda.gdn_chunk_fwd(*batch(on_gpu(x)), dpool, cu_seqlens=cu_of(lens, begin).cuda(),
                              slots=torch.full((4,), 9, dtype=torch.int32, device="cuda"))
    assert torch.equal(dpool, before)
    assert rel(o2[0, 5:172], reference(used, lens)[0]) <= TOL_O


@pytest.mark.gpu
def test_forward_neighbour_with_nan():
    """A sequence full of NaN leaves the one before it alone, whose last chunk reads into it."""
    lens = [40, 60]
    x = tokens(100, 1, 1, seed=22)
    for t in x[:3]:
        t[40:] = float("nan")
    ro, rS = reference([t[:40] for t in x], [40])
    o, S = kda.gdn_chunk_fwd(*batch(on_gpu(x)), cu_seqlens=cu_of(lens).cuda())
    assert rel(o[0, :40], ro) <= TOL_O and rel(S[0], rS[0]) <= TOL_S
    assert bool(torch.isnan(o[0, 40:]).all())


@pytest.mark.gpu
def test_forward_bad_offsets_are_contained():
    """Offsets that point outside or run backwards make empty or shortened sequences, nothing else."""
    x = tokens(100, 1, 2, seed=23)
    cu = torch.tensor([-50, 30, 20, 70, 1 << 30], dtype=torch.int32, device="cuda")
    o = torch.full((1, 100, 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    kda.gdn_chunk_fwd(*batch(on_gpu(x)), cu_seqlens=cu, o=o)
    torch.cuda.synchronize()
    assert kda.device_status() == kda.KDA_OK
    ro, _ = reference([t[:30] for t in x], [30])
    assert rel(o[0, :20], ro[:20]) <= TOL_O          # tokens 20-29 are in [0, 30) and [20, 70): either may be there


@pytest.mark.gpu
def test_forward_nothing_to_do():
    h = torch.randn(2, 2, D, D, device="cuda")
    e = [t.cuda() for t in batch(tokens(0, 1, 2, seed=1))]
    o, S = kda.gdn_chunk_fwd(*[t.expand(2, *t.shape[1:]).contiguous() for t in e], h)
    assert o.shape == (2, 0, 2, D) and torch.equal(S, h)
    o, S = kda.gdn_chunk_fwd(*e, cu_seqlens=torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert S.shape == (2, 2, D, D) and not S.any()
    o, S = kda.gdn_chunk_fwd(*e, cu_seqlens=torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert S.shape[0] == 0


@pytest.mark.gpu
def test_forward_repeats_and_captures():
    """Bitwise the same from run to run, on another stream and replayed from a graph."""
    lens = [300, 77]
    x = batch(on_gpu(tokens(377, 2, 4, seed=31)))
    cu = cu_of(lens).cuda()
    h = torch.randn(2, 4, D, D, device="cuda") * 0.1
    o, S = kda.gdn_chunk_fwd(*x, h, cu_seqlens=cu)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o1, S1 = kda.gdn_chunk_fwd(*x, h, cu_seqlens=cu)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, o1) and torch.equal(S, S1)
    o2, S2 = torch.zeros_like(o), torch.zeros_like(S)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            kda.gdn_chunk_fwd(*x, h, cu_seqlens=cu, o=o2, hT=S2)
        graphs.append(graph)
    for graph in graphs + graphs:
        o2.zero_(), S2.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(S, S2)


# ------------------------------------------------------------------ one token --

@pytest.mark.gpu
@pytest.mark.parametrize("dk", [32, 64, 128])
@pytest.mark.parametrize("dv", [32, 64, 128])
def test_step_shapes(dk, dv):
    for HK, HV, N in ((2, 4, 3), (1, 1, 1), (3, 3, 40)):
        x = tokens(N, HK, HV, seed=dk + dv + N, dk=dk, dv=dv, gate=torch.bfloat16 if N == 3 else torch.float32)
        S0 = torch.randn(N, HV, dk, dv, generator=torch.Generator().manual_seed(1)) * 0.3
        ro, rS = reference(x, [1] * N, S0, scale=0.5)
        S = S0.cuda()
        o = kda.gdn_decode_step(*on_gpu(x), S, scale=0.5)
        assert rel(o, ro) <= TOL_O
        assert rel(S, rS) <= TOL_STEP


@pytest.mark.gpu
def test_step_pool_and_padding():
    N, HV = 5, 4
    x = tokens(N, 2, HV, seed=41)
    pool = torch.randn(8, HV, D, D, generator=torch.Generator().manual_seed(2)) * 0.3
    slots = torch.tensor([6, -1, 0, 8, 3], dtype=torch.int32)
    real = [0, 2, 4]
    ro, rS = reference([t[real] for t in x], [1] * 3, pool[slots[real].long()])
    d = pool.cuda()
    o = kda.gdn_decode_step(*on_gpu(x), d, slots=slots.cuda())
    assert rel(o[real], ro) <= TOL_O and not o[[1, 3]].any()
    got = d.cpu()
    for r, n in ((6, 0), (0, 1), (3, 2)):
        assert rel(got[r], rS[n]) <= TOL_STEP
    for r in (1, 2, 4, 5, 7):
        assert torch.equal(got[r], pool[r])


@pytest.mark.gpu
def test_step_reset_and_nan():
    """A log-decay of -inf forgets the state; a NaN request leaves the others alone."""
    x = tokens(2, 1, 1, seed=42)
    x[3][0] = -torch.inf
    x[2][1] = float("nan")
    S = torch.randn(2, 1, D, D, device="cuda")
    o = kda.gdn_decode_step(*on_gpu(x), S)
    k, v, b = x[1][0, 0].double(), x[2][0, 0].double(), x[4][0, 0].double()
    assert rel(S[0, 0], b * k[:, None] * v[None]) <= TOL_STEP
    assert bool(torch.isnan(S[1]).any()) and bool(torch.isfinite(S[0]).all())
    assert rel(o[0, 0], b * (x[0][0, 0].double() @ k) * v) <= TOL_O


@pytest.mark.gpu
def test_prefill_then_decode():
    """A served request: prompts into a pool, then tokens one by one, against the whole sequence at once."""
    lens, more, HK, HV = [70, 5, 129], 6, 2, 4
    xs = [tokens(L + more, HK, HV, seed=50 + L) for L in lens]
    refs = [reference(x, [x[0].shape[0]], scale=0.1) for x in xs]
    pool = torch.zeros(4, HV, D, D, device="cuda")
    slots = torch.tensor([3, 0, 2], dtype=torch.int32, device="cuda")
    prompt = [torch.cat([x[i][:L] for x, L in zip(xs, lens)])[None].cuda() for i in range(5)]
    o, _ = kda.gdn_chunk_fwd(*prompt, pool, scale=0.1, cu_seqlens=cu_of(lens).cuda(), slots=slots)
    for n, (r, L) in enumerate(zip(refs, lens)):
        at = sum(lens[:n])
        assert rel(o[0, at:at + L], r[0][:L]) <= TOL_O
    for t in range(more):
        tok = [torch.stack([x[i][L + t] for x, L in zip(xs, lens)]).cuda() for i in range(5)]
        od = kda.gdn_decode_step(*tok, pool, scale=0.1, slots=slots)
        assert rel(od, np.stack([r[0][L + t] for r, L in zip(refs, lens)])) <= TOL_O
    assert rel(pool[slots.long()], np.concatenate([r[1] for r in refs])) <= TOL_S + more * TOL_STEP
