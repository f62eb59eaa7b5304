"""How many digits the gated delta rule with one decay per head keeps.

What the kernels compute and use again as an operand (S, U, T, W, P, and the
backward's dS, dU, dV, gam dO and pair gradients) is the sum of two bf16
numbers: hi is off by at most 2^-8 of the value, lo by at most 2^-8 of what hi
leaves, so a pair is off by at most 2^-16 of its value; the product lo lo, left
out, is at most 2^-16 as well.  Sums are fp32.  With n such errors in
quadrature, sqrt(n) 2^-16 bounds an fp32 output in the 2-norm:
  hT   T, -T diag(gam), W, S, W S without lo lo, U, eta U: 7;
       with segments the transition and the joined state as well: 9
  o    those, S again in Q S, P, U in P U, P U without lo lo: 11
  gradients  the forward's 7 in S0 and U, and dS, dU, dV, P, gam dO, W^T dU and
       dU^T T without lo lo, the pair gradients, the two products with states: 16
       (dg and dbeta take two gradients' worth: 32)
A bf16 output adds its own rounding.  Against the exact value that rounding
hides everything else (2^-8 / sqrt(3) in the norm), so outputs are compared
with the exact value ROUNDED to bf16: an error e then shows where it crosses a
border between two neighbours, a step of at most 2^-7 of the value, which
happens for |e| / step of the values.  The mean square of the difference is
step |e|, so with e in the norm of eps it is at most 2^-7 eps: sqrt(2^-7 eps),
and eps itself for what the borders do not catch.

A single bf16 in the place of any of those pairs is off by about 1.5e-3 and
must not pass: shown below on the host, with the same formulas in 64 bits.
"""
import numpy as np
import pytest
import torch

import linear_attention_07_b200 as kda
from test_gdn import D, batch, cu_of, on_gpu, rel, reference, tokens
from test_gdn_backward import cotangents, run
from test_gdn_backward import reference as gradients

PAIR = 2.0 ** -16
EPS_S, EPS_SEGMENTS, EPS_O, EPS_GRAD, EPS_GATE = (n ** 0.5 * PAIR for n in (7, 9, 11, 16, 32))
NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dh0")
EPS = (EPS_GRAD, EPS_GRAD, EPS_GRAD, EPS_GATE, EPS_GATE, EPS_GRAD)


def rounded(eps):
    return (2.0 ** -7 * eps) ** 0.5 + eps


def rel_rounded(x, ref):
    """Distance from the exact value as bf16 has it, in the norm of that."""
    return rel(x, torch.as_tensor(ref).to(torch.bfloat16).double())


# ------------------------------------------ the same formulas on the host, 64 bits --

C = 64


def pair(x):
    hi = x.to(torch.bfloat16).double()
    return hi + (x - hi).to(torch.bfloat16).double()


def single(x):
    return x.to(torch.bfloat16).double()


def by_chunks(x, h0, dO, dhT, scale, keep):
    """o, hT and the gradients of one head, chunk by chunk; keep(name, value) is what is kept of an operand."""
    q, k, v, g, beta = (t[:, 0].double() for t in x)
    dO, dS, S = dO[:, 0].double(), dhT.double(), h0.double()
    low, kept, o = torch.ones(C, C, dtype=torch.bool).tril(), [], []
    eye = torch.eye(C, dtype=torch.float64)
    for at in range(0, len(q), C):
        Q, K, V, b = q[at:at + C], k[at:at + C], v[at:at + C], beta[at:at + C]
        G = g[at:at + C].cumsum(0)
        gam, eta = G.exp()[:, None], (G[-1] - G).exp()[:, None]
        decay = torch.where(low, G[:, None] - G[None], -torch.inf).exp()
        T = torch.linalg.inv(eye + torch.where(low & (eye == 0), b[:, None] * decay * (K @ K.T), 0.0)) * b
        W = keep("W", keep("T gam", T * gam.T) @ K)
        P, T, S0 = keep("P", scale * decay * (Q @ K.T)), keep("T", T), keep("S", S)
        U = T @ V - W @ S0
        o.append(scale * gam * (Q @ S0) + P @ keep("U", U))
        S = gam[-1] * S + K.T @ keep("eta U", eta * U)
        kept.append((at, Q, K, b, gam, eta, decay, T, W, P, S0, keep("U kept", U)))
    last, out = S, [torch.zeros_like(t) for t in (q, k, v, g, beta)]
    for at, Q, K, b, gam, eta, decay, T, W, P, S0, U in reversed(kept):
        here, d = slice(at, at + C), dO[at:at + C]
        dS1 = keep("dS", dS)
        dU = keep("dU", P.T @ d + eta * (K @ dS1))
        gdO = keep("gam dO", scale * gam * d)
        dV = T.T @ dU
        dV2 = keep("dV", dV)
        dkk = keep("dkk", -decay * torch.where(eye == 0, dV2 @ U.T, 0.0))
        dqk = keep("dqk", scale * decay * (d @ U.T))
        out[0][here] = gam * scale * (d @ S0.T) + dqk @ K
        out[1][here] = -gam * (dV2 @ S0.T) + eta * (U @ dS1.T) + (dkk + dkk.T) @ K + dqk.T @ Q
        out[2][here] = dV
        a = (gam * ((scale * d) * (Q @ S0) - dV2 * (K @ S0))).sum(1)
        w = dqk * (Q @ K.T) + dkk * (K @ K.T)
        b_ = (eta * U * (K @ dS1)).sum(1)
        cross = torch.stack([w[t:, :t].sum() for t in range(C)])
        out[3][here] = gam[-1] * (dS1 * S0).sum() + a.flip(0).cumsum(0).flip(0) + b_.cumsum(0) - b_ + cross
        out[4][here] = (dV2 * U).sum(1) / b ** 2
        dS = gam[-1] * dS - W.T @ dU + Q.T @ gdO
    return torch.cat(o), last, out + [dS]


def host_errors(decay, keep):
    T, scale = 6 * C, 0.3
    x = tokens(T, 1, 1, seed=3, decay=decay)
    dO, dhT = cotangents(T, 1, 1)
    h0 = torch.randn(D, D, generator=torch.Generator().manual_seed(4))
    got = by_chunks(x, h0, dO, dhT[0, 0], scale, keep)
    ro, rS = reference(x, [T], h0[None, None], scale=scale)
    want = gradients(x, [T], dO, h0[None, None], dhT, scale=scale)
    errors = [rel_rounded(got[0].to(torch.bfloat16), ro[:, 0]) / rounded(EPS_O), rel(got[1], rS[0, 0]) / EPS_S]
    for a, b, eps in zip(got[2][:5], want, EPS):
        errors.append(rel_rounded(a.to(torch.bfloat16), b[:, 0]) / rounded(eps))
    return errors + [rel(got[2][5], want[5][0, 0]) / EPS_GRAD]


@pytest.mark.parametrize("decay", ["trained", "none", "strong"])
def test_pairs_are_within_the_bounds(decay):
    assert max(host_errors(decay, lambda name, x: pair(x))) <= 1


@pytest.mark.parametrize("lost", ["T gam", "W", "P", "T", "S", "U", "eta U", "U kept", "dS", "dU", "dV", "dkk", "dqk", "gam dO"])
def test_a_lost_lower_plane_is_seen(lost):
    """A single bf16 in the place of one pair fails the bounds."""
    assert max(host_errors("none", lambda name, x: single(x) if name == lost else pair(x))) > 1.5


# ---------------------------------------------------------------- the kernels --

@pytest.mark.gpu
@pytest.mark.parametrize("decay", ["trained", "none", "strong", "far", "reset"])
@pytest.mark.parametrize("lens", [(200, 1, 64, 333), (700,)], ids=str)
def test_forward_digits(decay, lens):
    x = tokens(sum(lens), 2, 4, seed=61, decay=decay)
    ref = list(x)
    ref[3] = torch.clamp(x[3], min=-1e4)
    h0 = torch.randn(len(lens), 4, D, D, generator=torch.Generator().manual_seed(62))
    ro, rS = reference(ref, lens, h0, scale=0.3)
    o, S = kda.gdn_chunk_fwd(*batch(on_gpu(x)), h0.cuda(), scale=0.3, cu_seqlens=cu_of(lens).cuda())
    assert rel_rounded(o[0], ro) <= rounded(EPS_O) and rel(S, rS) <= EPS_S


@pytest.mark.gpu
@pytest.mark.parametrize("decay", ["trained", "none", "strong", "far", "reset"])
@pytest.mark.parametrize("lens", [(200, 1, 64, 333), (700,)], ids=str)
def test_gradient_digits(decay, lens):
    x = tokens(sum(lens), 2, 4, seed=63, decay=decay)
    ref = list(x)
    ref[3] = torch.clamp(x[3], min=-1e4)
    dO, dhT = cotangents(sum(lens), 4, len(lens))
    h0 = torch.randn(len(lens), 4, D, D, generator=torch.Generator().manual_seed(64))
    got, want = run(x, lens, dO, h0, dhT, scale=0.3), gradients(ref, lens, dO, h0, dhT, scale=0.3)
    errors = {name: (rel_rounded(a[0], b), rounded(eps)) for name, a, b, eps in zip(NAMES[:5], got, want, EPS)}
    errors["dh0"] = rel(got[5], want[5]), EPS_GRAD
    assert all(e <= t for e, t in errors.values()), errors


@pytest.mark.gpu
@pytest.mark.parametrize("decay", ["trained", "strong", "far", "reset"])
def test_digits_in_segments(decay):
    """Transitions that become zero, or that resets cut, among them."""
    lens, HV = (2600, 0, 2100), 4
    x = tokens(sum(lens), 2, HV, seed=65, decay=decay)
    ref = list(x)
    ref[3] = torch.clamp(x[3], min=-1e4)
    dO, dhT = cotangents(sum(lens), HV, len(lens))
    h0 = torch.randn(len(lens), HV, D, D, generator=torch.Generator().manual_seed(66))
    n0 = kda.launch_count()
    o, S = kda.gdn_chunk_fwd(*batch(on_gpu(x)), h0.cuda(), cu_seqlens=cu_of(lens).cuda())
    assert kda.launch_count() - n0 == 2                  # 24 chunks on average: in one piece
    lens = (4700,)
    h0, dhT = h0[:1], dhT[:1]
    n0 = kda.launch_count()
    o, S = kda.gdn_chunk_fwd(*batch(on_gpu(x)), h0.cuda(), cu_seqlens=cu_of(lens).cuda())
    assert kda.launch_count() - n0 == 4
    ro, rS = reference(ref, lens, h0)
    assert rel_rounded(o[0], ro) <= rounded(EPS_O) and rel(S, rS) <= EPS_SEGMENTS
    got, want = run(x, lens, dO, h0, dhT), gradients(ref, lens, dO, h0, dhT)
    errors = {name: (rel_rounded(a[0], b), rounded(eps)) for name, a, b, eps in zip(NAMES[:5], got, want, EPS)}
    errors["dh0"] = rel(got[5], want[5]), EPS_GRAD
    assert all(e <= t for e, t in errors.values()), errors
