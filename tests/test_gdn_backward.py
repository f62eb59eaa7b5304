"""Backward of the gated delta rule with one decay per head
(kda_gdn_chunk_bwd, kda_gdn_chunk_bwd_packed8) against the fp64 backward oracle
(per-channel decay, so dg is the sum over the channels; dq and dk of a shared
head are the sums over its value heads).

Tolerances.  One rounding to bf16 is off by 2^-8 at most, 2^-8 / sqrt(3) in
the root mean square.  These bounds leave room for four of them in quadrature,
2 * 2^-8 / sqrt(3) (TOL_GRAD), and for dg, a sum over up to 64 tokens, sqrt(64)
as much (TOL_DG); the kernels round to bf16 once, at the end, and what their
pairs of bf16 keep is held in test_gdn_digits.py.  dh0 is fp32 through pairs of bf16, as the forward's state.
"""
import numpy as np
import pytest
import torch

import linear_attention_07_b200 as kda
from test_gdn import D, TOL_S, batch, cu_of, on_gpu, rel, tokens

TOL_GRAD = 2 * 2.0 ** -8 / 3 ** 0.5
TOL_DG = 8 * TOL_GRAD


def reference(x, lens, dO, h0=None, dhT=None, scale=1.0, begin=0):
    import oracle
    q, k, v, g, b = (t.double() for t in x)
    T, HK, dk = q.shape
    HV, dv = v.shape[1:]
    r = HV // HK
    q, k = (t.repeat_interleave(r, 1) for t in (q * scale, k))
    gc = g[..., None].expand(T, HV, dk)
    out = [np.zeros((T, HV, dk)), np.zeros((T, HV, dk)), np.zeros((T, HV, dv)), np.zeros((T, HV)), np.zeros((T, HV))]
    dh0 = np.zeros((len(lens), HV, dk, dv))
    at = begin
    for n, L in enumerate(lens):
        sl = slice(at, at + L)
        at += L
        h = None if h0 is None else h0[n:n + 1]
        dh = None if dhT is None else dhT[n:n + 1]
        if not L:
            dh0[n] = 0 if dh is None else dh[0].double().numpy()
            continue
        got = oracle.bwd(*(t[None, sl] for t in (q, k, v, gc, b)), h, dO[None, sl].double(), dh)
        got[0][:] *= scale
        for i in range(5):
            out[i][sl] = got[i][0].sum(-1) if i == 3 else got[i][0]
        dh0[n] = got[5][0]
    for i in range(2):
        out[i] = out[i].reshape(T, HK, r, dk).sum(2)
    return out + [dh0]


def cotangents(T, HV, N, seed=9):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(T, HV, D, generator=gen).to(torch.bfloat16), torch.randn(N, HV, D, D, generator=gen) * 0.1


def check(got, want, tols=(TOL_GRAD, TOL_GRAD, TOL_GRAD, TOL_DG, TOL_GRAD, TOL_S)):
    errors = {}
    for name, x, y, tol in zip(("dq", "dk", "dv", "dg", "dbeta", "dh0"), got, want, tols):
        if x is not None:
            errors[name] = (rel(x[0] if name != "dh0" else x, y), tol)
    assert all(e <= t for e, t in errors.values()), errors
    assert kda.device_status() == kda.KDA_OK


def run(x, lens, dO, h0=None, dhT=None, **kw):
    dev = lambda t: None if t is None else t.cuda()
    return kda.gdn_chunk_bwd(*batch(on_gpu(x)), dev(h0), dO[None].cuda(), dev(dhT), cu_seqlens=cu_of(lens).cuda(), **kw)


def test_refusals_on_the_host():
    import ctypes
    lib = kda.load_library()
    n0 = lib.kda_launch_count()
    A, MIS, NUL = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008), None

    def bwd(q=A, dO=A, dhT=NUL, dq=A, dk=A, dv=A, dg=A, dbeta=A, dh0=A, cu=NUL, N=1, T=64, HK=2, HV=4, d_k=128, d_v=128,
            qs=256, g=A):
        return lib.kda_gdn_chunk_bwd(q, A, A, g, A, NUL, dO, dhT, dq, dk, dv, dg, dbeta, dh0, cu, 1.0, N, T, HK, HV, d_k,
                                     d_v, qs, 256, 512, 1, None)

    for bad in (dict(q=NUL), dict(dO=NUL), dict(dO=MIS), dict(dq=NUL), dict(dk=MIS), dict(dv=NUL), dict(dg=NUL),
                dict(dbeta=NUL), dict(dh0=MIS), dict(dhT=MIS), dict(T=-1), dict(HK=3), dict(qs=128), dict(g=NUL),
                dict(dg=ctypes.c_void_p(0x10001))):
        assert bwd(**bad) == kda.KDA_ERR_INVALID_ARG, bad
    assert bwd(d_k=64, qs=256) == kda.KDA_ERR_UNSUPPORTED
    assert bwd(N=0) == kda.KDA_OK and bwd(T=0, dh0=NUL) == kda.KDA_OK

    def packed(qs=A, d_k=128, dO=A):
        return lib.kda_gdn_chunk_bwd_packed8(A, A, A, qs, A, A, A, A, NUL, dO, NUL, A, A, A, A, A, A, NUL, 1.0, 1, 64, 2, 4,
                                             d_k, 128, 1, None)

    assert packed(qs=NUL) == kda.KDA_ERR_INVALID_ARG and packed(dO=NUL) == kda.KDA_ERR_INVALID_ARG
    assert packed(d_k=64) == kda.KDA_ERR_UNSUPPORTED
    assert lib.kda_launch_count() == n0
    x = batch(tokens(4, 2, 4, seed=0))
    with pytest.raises(ValueError, match="CUDA"):
        kda.gdn_chunk_bwd(*x, None, x[2])
    p = kda.Packed8(torch.zeros(1, 4, 2, 128, dtype=torch.float8_e4m3fn), torch.zeros(1, 4, 2, 4, dtype=torch.uint8))
    with pytest.raises(TypeError, match="Packed8"):
        kda.gdn_chunk_bwd(p, *x[1:], None, x[2])


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [(1,), (2, 1), (16, 17), (63, 64, 65), (127, 0, 128, 129), (200, 1, 1, 333)], ids=str)
@pytest.mark.parametrize("ends", [False, True])
def test_ragged(lens, ends):
    HK, HV = 2, 4
    for gate in (torch.float32, torch.bfloat16):
        x = tokens(sum(lens), HK, HV, seed=sum(lens) + 3, gate=gate)
        dO, dhT = cotangents(sum(lens), HV, len(lens))
        h0 = torch.randn(len(lens), HV, D, D, generator=torch.Generator().manual_seed(3)) * 0.1 if ends else None
        dhT = dhT if ends else None
        check(run(x, lens, dO, h0, dhT, scale=0.3), reference(x, lens, dO, h0, dhT, scale=0.3))


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [(1, 1), (3, 3), (2, 10)], ids=str)
def test_heads_in_a_batch(heads):
    HK, HV = heads
    B, T = 2, 100
    x = tokens(B * T, HK, HV, seed=HV)
    dO, _ = cotangents(B * T, HV, B)
    want = reference(x, [T] * B, dO)
    y = [t.reshape(B, T, *t.shape[1:]).contiguous().cuda() for t in x]
    got = kda.gdn_chunk_bwd(*y, None, dO.reshape(B, T, HV, D).cuda())
    check([t.flatten(0, 1)[None] for t in got[:5]] + [got[5]], want)
    assert kda.gdn_chunk_bwd(*y, None, dO.reshape(B, T, HV, D).cuda(), want_dh0=False)[5] is None


@pytest.mark.gpu
@pytest.mark.parametrize("decay", ["none", "strong", "reset"])
def test_decays(decay):
    x = tokens(200, 1, 2, seed=11, decay=decay)
    ref = list(x)
    ref[3] = torch.clamp(x[3], min=-1e4)
    dO, dhT = cotangents(200, 2, 1)
    h0 = torch.randn(1, 2, D, D, generator=torch.Generator().manual_seed(4)) * 0.1
    check(run(x, [200], dO, h0, dhT), reference(ref, [200], dO, h0, dhT))


@pytest.mark.gpu
@pytest.mark.parametrize("decay", ["trained", "strong", "far", "reset"])
def test_linear_in_values_and_cotangents(decay):
    """Gradients of powers of two times (v, h0) or (dO, dhT): dq, dk, dg and dbeta take both factors, dv and dh0 the
    cotangents' only, and no bit changes (numbers 2^-60 below the largest aside)."""
    lens = [150, 65, 1, 64]
    T = sum(lens)
    x = tokens(T, 2, 4, seed=17, decay=decay)
    dO, dhT = cotangents(T, 4, len(lens))
    h0 = torch.randn(len(lens), 4, D, D, generator=torch.Generator().manual_seed(7))
    want = [t.double() for t in run(x, lens, dO, h0, dhT)]
    for ev, eo in ((-30, 0), (30, 0), (0, -30), (0, 30)):
        fv, fo = 2.0 ** ev, 2.0 ** eo
        y = list(on_gpu(x))
        y[2].copy_(y[2] * fv)
        got = kda.gdn_chunk_bwd(*batch(y), (h0 * fv).cuda(), (dO * fo)[None].cuda(), (dhT * fo).cuda(), cu_seqlens=cu_of(lens).cuda())
        for name, a, b in zip(("dq", "dk", "dv", "dg", "dbeta", "dh0"), got, want):
            a = a.double() / (fo if name in ("dv", "dh0") else fv * fo)
            counts = b.abs() >= b.abs().max() * 2.0 ** -60
            assert torch.equal(a[counts], b[counts]), (name, ev, eo)
    assert kda.device_status() == kda.KDA_OK


@pytest.mark.gpu
@pytest.mark.parametrize("beta", [0.0, 1e-12, 1.0])
def test_write_strengths(beta):
    """beta = 0 writes nothing, yet its own gradient is not zero."""
    x = tokens(130, 1, 2, seed=12, beta=beta)
    dO, dhT = cotangents(130, 2, 1)
    h0 = torch.randn(1, 2, D, D, generator=torch.Generator().manual_seed(4)) * 0.1
    got, want = run(x, [130], dO, h0, dhT), reference(x, [130], dO, h0, dhT)
    # terms in beta are 2^-30 where they should be 0 or 1e-12
    check([t if i not in (1, 2) else None for i, t in enumerate(got)], want)
    for i in (1, 2):
        err = np.linalg.norm(got[i][0].double().cpu().numpy() - want[i])
        assert err <= TOL_GRAD * np.linalg.norm(want[i]) + 2.0 ** -28 * np.sqrt(want[i].size)


@pytest.mark.gpu
def test_differences():
    """The gradients against differences of the forward (fp64), along the gradients' own direction."""
    from test_gdn import reference as forward
    lens = [150]
    x = tokens(150, 1, 2, seed=14)
    dO, dhT = cotangents(150, 2, 1)
    h0 = torch.randn(1, 2, D, D, generator=torch.Generator().manual_seed(5)) * 0.1
    got = [t.double().cpu() for t in run(x, lens, dO, h0, dhT, scale=0.5)]
    grads = [t[0] for t in got[:5]] + [got[5]]
    at = [t.double() for t in x] + [h0.double()]

    def loss(eps, i):
        y = [t + (eps * grads[i] / grads[i].norm() if n == i else 0) for n, t in enumerate(at)]
        o, S = forward(y[:5], lens, y[5], scale=0.5)
        return float((torch.from_numpy(o) * dO.double()).sum() + (torch.from_numpy(S) * dhT.double()).sum())

    for i, tol in enumerate((TOL_GRAD, TOL_GRAD, TOL_GRAD, TOL_DG, TOL_GRAD, TOL_S)):
        eps = 1e-4                                     # the difference's own error: eps^2 relative
        slope = (loss(eps, i) - loss(-eps, i)) / (2 * eps)
        assert abs(slope - float(grads[i].norm())) <= 2 * tol * abs(slope), (i, slope, float(grads[i].norm()))


@pytest.mark.gpu
def test_long_and_repeatable():
    x = tokens(3000, 2, 2, seed=15)
    dO, dhT = cotangents(3000, 2, 1)
    got = run(x, [3000], dO, None, dhT)
    check(got, reference(x, [3000], dO, None, dhT))
    again = run(x, [3000], dO, None, dhT)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.gpu
def test_tokens_outside_and_neighbours():
    """Tokens of no sequence get zero gradients, and what they or a neighbour hold goes nowhere else."""
    lens, begin, T = [70, 0, 33], 5, 160
    x = tokens(T, 2, 4, seed=21)
    dO, _ = cotangents(T, 4, 3)
    for t in (*x[:3], dO):
        t[:5] = float("nan")
        t[75:108] = float("nan")                       # the last sequence, and
        t[108:] = float("inf")                         # what comes behind it
    used = [t[5:75] for t in x]
    want = reference(used, [70], dO[5:75])
    cu = cu_of(lens, begin).cuda()
    got = kda.gdn_chunk_bwd(*batch(on_gpu(x)), None, dO[None].cuda(), cu_seqlens=cu)
    check([t[:, 5:75] for t in got[:5]] + [got[5][:1]], want)
    for t in got[:5]:
        assert not t[0, :5].any() and not t[0, 108:].any()
    assert not got[5][1].any()
    none = kda.gdn_chunk_bwd(*batch(on_gpu(x)), None, dO[None].cuda(), cu_seqlens=torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert not any(bool(t.any()) for t in none[:5])


@pytest.mark.gpu
def test_bad_offsets_are_contained():
    x = tokens(100, 1, 2, seed=23)
    dO, _ = cotangents(100, 2, 4)
    cu = torch.tensor([-50, 30, 20, 70, 1 << 30], dtype=torch.int32, device="cuda")
    kda.gdn_chunk_bwd(*batch(on_gpu(x)), None, dO[None].cuda(), cu_seqlens=cu)
    torch.cuda.synchronize()
    assert kda.device_status() == kda.KDA_OK


@pytest.mark.gpu
def test_no_tokens():
    e = [t.cuda() for t in batch(tokens(0, 1, 2, seed=1))]
    dhT = torch.randn(2, 2, D, D, device="cuda")
    e2 = [t.expand(2, *t.shape[1:]).contiguous() for t in e]
    got = kda.gdn_chunk_bwd(*e2, None, e2[2], dhT)
    assert torch.equal(got[5], dhT) and got[0].shape == (2, 0, 1, D)
    assert not kda.gdn_chunk_bwd(*e2, None, e2[2])[5].any()


@pytest.mark.gpu
def test_from_8_bits():
    """The backward from 8-bit checkpoints is, bit for bit, the backward of the values they stand for."""
    lens = [100, 65]
    x = on_gpu(tokens(165, 2, 4, seed=31))
    dO, dhT = cotangents(165, 4, 2)
    q, k, v, g, b = batch(x)
    packed = kda.act_pack8(q, k, v)
    cu = cu_of(lens).cuda()
    got = kda.gdn_chunk_bwd(*packed, g, b, None, dO[None].cuda(), dhT.cuda(), cu_seqlens=cu)
    vals = [kda.act_unpack8(p) for p in packed]
    want = kda.gdn_chunk_bwd(*vals, g, b, None, dO[None].cuda(), dhT.cuda(), cu_seqlens=cu)
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    ref = reference([t[0].cpu() for t in vals] + [x[3].cpu(), x[4].cpu()], lens, dO, None, dhT)
    check(got, ref)


@pytest.mark.gpu
def test_training_step_in_a_graph():
    """Forward, checkpoint, backward as a training step runs them, captured while an eager graph of the same leaves lives."""
    x = batch(on_gpu(tokens(200, 2, 4, seed=41)))
    cu = cu_of([120, 80]).cuda()
    dO, dhT = cotangents(200, 4, 2)
    dO, dhT = dO[None].cuda(), dhT.cuda()

    def step():
        o, S = kda.gdn_chunk_fwd(*x, cu_seqlens=cu)
        packed = kda.act_pack8(*x[:3])
        return (o, S) + kda.gdn_chunk_bwd(*packed, *x[3:], None, dO, dhT, cu_seqlens=cu)

    want = step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
