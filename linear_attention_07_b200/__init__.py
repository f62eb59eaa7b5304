"""Kimi Delta Attention (KDA) prefill and decode on NVIDIA B200 (sm_100a).

Thin ctypes binding over ``libkda.so`` (the C ABI declared in
``include/kda.h``).  Every step of the computation runs in the library's
CUDA kernels; this module only checks tensors and passes pointers, sizes
and the current CUDA stream of the tensors' device, which it makes the
current device for the call.  PyTorch is used for device memory and streams.

Raw C functions are exposed under their C names (every name in
``EXPORTED``).  The tensor-level helpers wrap them: ``chunk_fwd``,
``chunk_fwd_raw`` (prologue fused), ``chunk_fwd_noalloc``,
``chunk_fwd_states`` (intermediate states), ``chunk_transition`` and
``state_chain`` (the pieces of a split sequence), ``chunk_fwd_f32``,
``decode_step``, ``decode_step_raw``, ``verify_fwd`` (several tokens
per request with the state after each) and ``chunk_bwd`` (the gradients).  They accept only contiguous CUDA
tensors of the documented dtypes and shapes.

The gated delta rule with one decay per head: ``gdn_chunk_fwd`` (packed
sequences, grouped heads, pools of states), ``gdn_chunk_bwd`` and
``gdn_decode_step``; their q, k and v may be slices of one projection's
output.  ``act_pack8`` and ``act_unpack8`` keep activations in 8 bits
(``Packed8``), which ``gdn_chunk_bwd`` also takes as they are.

If the library is missing or cannot be loaded, every call raises
``KdaLibraryError``: there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libkda.so")

KDA_OK = 0
KDA_ERR_INVALID_ARG = -1
KDA_ERR_UNSUPPORTED = -2
KDA_ERR_CUDA = -3
KDA_ERR_TIMEOUT = -4
KDA_ERR_NO_MEMORY = -5

EXPORTED = ("kda_chunk_fwd", "kda_chunk_fwd_noalloc", "kda_chunk_fwd_states", "kda_chunk_fwd_f32",
            "kda_chunk_transition", "kda_state_chain", "kda_chunk_fwd_raw", "kda_decode_step",
            "kda_decode_step_raw", "kda_verify_fwd", "kda_chunk_bwd", "kda_chunk_bwd_raw",
            "kda_gdn_chunk_fwd", "kda_gdn_chunk_bwd", "kda_gdn_chunk_bwd_packed8", "kda_gdn_decode_step",
            "kda_act_pack8", "kda_act_unpack8",
            "kda_device_status", "kda_selftest_bounded_wait",
            "kda_status_string", "kda_launch_count", "kda_prefill_path", "kda_version")


class KdaLibraryError(RuntimeError):
    pass


class KdaError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__("%s failed: %s (%d)" % (fn, status_string(status), status))


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libkda.so (once) and declare the C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise KdaLibraryError(
            "libkda.so not found at %s; build it with "
            "`python -m linear_attention_07_b200.build`" % path)
    try:
        lib = ctypes.CDLL(path)
    except OSError as e:  # pragma: no cover - depends on the machine
        raise KdaLibraryError("cannot load %s: %s" % (path, e)) from e
    vp, fp, i = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int
    lib.kda_chunk_fwd.argtypes = [vp, vp, vp, vp, vp, fp, vp, fp, i, i, i, i, i, vp]
    lib.kda_chunk_fwd.restype = i
    lib.kda_chunk_fwd_noalloc.argtypes = [vp, vp, vp, vp, vp, fp, vp, fp, i, i, i, i, i, vp]
    lib.kda_chunk_fwd_noalloc.restype = i
    lib.kda_chunk_fwd_states.argtypes = [vp, vp, vp, vp, vp, fp, vp, fp, fp, i, i, i, i, i, i, vp]
    lib.kda_chunk_fwd_states.restype = i
    lib.kda_chunk_transition.argtypes = [vp, vp, vp, vp, fp, i, i, i, i, vp]
    lib.kda_chunk_transition.restype = i
    lib.kda_state_chain.argtypes = [fp, fp, fp, fp, fp, i, i, i, i, i, vp]
    lib.kda_state_chain.restype = i
    lib.kda_chunk_fwd_f32.argtypes = [fp, fp, fp, fp, fp, fp, fp, fp, i, i, i, i, i, vp]
    lib.kda_chunk_fwd_f32.restype = i
    lib.kda_decode_step.argtypes = [vp, vp, vp, vp, vp, fp, vp, i, i, i, i, vp]
    lib.kda_decode_step.restype = i
    lib.kda_chunk_fwd_raw.argtypes = [vp, vp, vp, vp, vp, fp, vp, fp, i, i, i, i, i, vp]
    lib.kda_chunk_fwd_raw.restype = i
    lib.kda_decode_step_raw.argtypes = [vp, vp, vp, vp, vp, fp, vp, i, i, i, i, vp]
    lib.kda_decode_step_raw.restype = i
    lib.kda_chunk_bwd.argtypes = [vp, vp, vp, vp, vp, fp, vp, fp, vp, vp, vp, vp, vp, fp,
                                  i, i, i, i, i, vp]
    lib.kda_chunk_bwd.restype = i
    lib.kda_chunk_bwd_raw.argtypes = lib.kda_chunk_bwd.argtypes
    lib.kda_chunk_bwd_raw.restype = i
    lib.kda_verify_fwd.argtypes = [vp, vp, vp, vp, vp, fp, vp, fp, i, i, i, i, i, vp]
    lib.kda_verify_fwd.restype = i
    i64, f = ctypes.c_int64, ctypes.c_float
    lib.kda_gdn_decode_step.argtypes = [vp, vp, vp, vp, vp, fp, vp, vp, i, f, i, i, i, i, i, i64, i64, i64, i, vp]
    lib.kda_gdn_decode_step.restype = i
    lib.kda_gdn_chunk_fwd.argtypes = [vp, vp, vp, vp, vp, fp, vp, fp, vp, vp, i, f, i, i, i, i, i, i, i64, i64, i64, i, vp]
    lib.kda_gdn_chunk_fwd.restype = i
    lib.kda_gdn_chunk_bwd.argtypes = [vp] * 14 + [vp, f, i, i, i, i, i, i, i64, i64, i64, i, vp]
    lib.kda_gdn_chunk_bwd.restype = i
    lib.kda_gdn_chunk_bwd_packed8.argtypes = [vp] * 17 + [vp, f, i, i, i, i, i, i, i, vp]
    lib.kda_gdn_chunk_bwd_packed8.restype = i
    lib.kda_act_pack8.argtypes = [i, vp, vp, vp, vp, vp, vp, vp]
    lib.kda_act_pack8.restype = i
    lib.kda_act_unpack8.argtypes = [i, vp, vp, vp, vp, vp, vp]
    lib.kda_act_unpack8.restype = i
    lib.kda_device_status.argtypes = [vp]
    lib.kda_device_status.restype = i
    lib.kda_selftest_bounded_wait.argtypes = [ctypes.c_uint64, vp]
    lib.kda_selftest_bounded_wait.restype = i
    lib.kda_status_string.argtypes = [i]
    lib.kda_status_string.restype = ctypes.c_char_p
    lib.kda_launch_count.argtypes = []
    lib.kda_launch_count.restype = ctypes.c_uint64
    lib.kda_prefill_path.argtypes = [i, i, i]
    lib.kda_prefill_path.restype = i
    lib.kda_version.argtypes = []
    lib.kda_version.restype = i
    _lib = lib
    return lib


def __getattr__(name):
    # raw C entry points under their C names, resolved on first use
    if name in EXPORTED:
        return getattr(load_library(), name)
    raise AttributeError(name)


def status_string(status: int) -> str:
    return load_library().kda_status_string(int(status)).decode()


def device_status(device=None) -> int:
    """KDA_OK or KDA_ERR_TIMEOUT (a bounded device wait expired since the
    last call); synchronises the current stream and clears the flag."""
    import torch
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(dev):
        return int(load_library().kda_device_status(_stream(dev)))


PREFILL_PATHS = ("one SM per head", "cluster of four SMs per head", "segment scan")


def prefill_path(B: int, T: int, H: int) -> str:
    """The path a bf16 prefill of this shape takes on the current device."""
    p = int(load_library().kda_prefill_path(int(B), int(T), int(H)))
    if p < 0:
        raise KdaError("kda_prefill_path", p)
    return PREFILL_PATHS[p]


def launch_count() -> int:
    """Kernels launched by libkda.so so far in this process."""
    return int(load_library().kda_launch_count())


# ---------------------------------------------------------------- tensors --

def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device):
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _require_cuda(t, name="inputs"):
    if t.device.type != "cuda":
        raise ValueError("%s must be CUDA tensors, got %s" % (name, t.device))
    return t.device


def _check(t, name, dtype, shape, device):
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.device != device:
        raise ValueError("%s must be on %s, got %s" % (name, device, t.device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _prefill(fn_name, dtype, q, k, v, g, beta, h0, o, hT, output_final_state):
    import torch
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dev = _require_cuda(q)
    for name, t, shp in (("q", q, (B, T, H, dk)), ("k", k, (B, T, H, dk)),
                         ("g", g, (B, T, H, dk)), ("v", v, (B, T, H, dv)),
                         ("beta", beta, (B, T, H))):
        _check(t, name, dtype, shp, dev)
    if h0 is not None:
        _check(h0, "h0", torch.float32, (B, H, dk, dv), dev)
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=dtype, device=dev)
    _check(o, "o", dtype, (B, T, H, dv), dev)
    if hT is None and output_final_state:
        hT = torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev)
    if hT is not None:
        _check(hT, "hT", torch.float32, (B, H, dk, dv), dev)
    fn = getattr(load_library(), fn_name)
    with torch.cuda.device(dev):
        st = fn(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0), _ptr(o),
                _ptr(hT), B, T, H, dk, dv, _stream(dev))
    if st != KDA_OK:
        raise KdaError(fn_name, st)
    return o, hT


def chunk_fwd(q, k, v, g, beta, h0=None, *, o=None, hT=None, output_final_state=True):
    """KDA prefill, bf16 in/out, fp32 state (kda_chunk_fwd).

    q, k, g: [B, T, H, dk]; v: [B, T, H, dv]; beta: [B, T, H] (bf16, CUDA,
    contiguous); h0: [B, H, dk, dv] fp32 or None.  Returns (o, hT).
    hT may be passed as h0 to update a state in place.
    """
    import torch
    return _prefill("kda_chunk_fwd", torch.bfloat16, q, k, v, g, beta, h0, o,
                    hT, output_final_state)


def chunk_fwd_raw(q_raw, k_raw, v, z, beta, h0=None, *, o=None, hT=None, output_final_state=True):
    """chunk_fwd with the prologue fused in (kda_chunk_fwd_raw): q_raw, k_raw
    unnormalised, z the gate pre-activation (g = -5 sigmoid(z) in the kernel)."""
    import torch
    return _prefill("kda_chunk_fwd_raw", torch.bfloat16, q_raw, k_raw, v, z, beta, h0, o,
                    hT, output_final_state)


def chunk_fwd_noalloc(q, k, v, g, beta, h0=None, *, o=None, hT=None, output_final_state=True):
    """chunk_fwd without any allocation in the library (kda_chunk_fwd_noalloc):
    the segment-scan path uses the library's fixed device scratch."""
    import torch
    return _prefill("kda_chunk_fwd_noalloc", torch.bfloat16, q, k, v, g, beta, h0, o,
                    hT, output_final_state)


def chunk_fwd_states(q, k, v, g, beta, h0=None, *, state_every, o=None, hT=None, states=None):
    """chunk_fwd that also returns the fp32 state after every `state_every`
    tokens (kda_chunk_fwd_states): (o, hT, states), states [B, H, T //
    state_every, dk, dv]."""
    import torch
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    _require_cuda(q)
    n = T // state_every if state_every > 0 else 0
    if states is None:
        states = torch.empty((B, H, n, dk, dv), dtype=torch.float32, device=q.device)
    _check(states, "states", torch.float32, (B, H, n, dk, dv), q.device)
    if o is None:
        o = torch.empty_like(v)
    if hT is None:
        hT = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    for name, t, shp in (("q", q, (B, T, H, dk)), ("k", k, (B, T, H, dk)), ("g", g, (B, T, H, dk)),
                         ("v", v, (B, T, H, dv)), ("beta", beta, (B, T, H)), ("o", o, (B, T, H, dv))):
        _check(t, name, torch.bfloat16, shp, q.device)
    _check(hT, "hT", torch.float32, (B, H, dk, dv), q.device)
    if h0 is not None:
        _check(h0, "h0", torch.float32, (B, H, dk, dv), q.device)
    with torch.cuda.device(q.device):
        st = load_library().kda_chunk_fwd_states(
            _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0), _ptr(o), _ptr(hT),
            _ptr(states) if n > 0 else None, int(state_every), B, T, H, dk, dv,
            _stream(q.device))
    if st != KDA_OK:
        raise KdaError("kda_chunk_fwd_states", st)
    return o, hT, states


def chunk_transition(q, k, g, beta, *, M=None):
    """Transition M [B, H, dk, dk] (fp32) of each whole sequence
    (kda_chunk_transition): running it from S0 ends at M S0 + (its state from zero)."""
    import torch
    B, T, H, dk = q.shape
    dev = _require_cuda(q)
    for name, t, shp in (("q", q, (B, T, H, dk)), ("k", k, (B, T, H, dk)), ("g", g, (B, T, H, dk)),
                         ("beta", beta, (B, T, H))):
        _check(t, name, torch.bfloat16, shp, dev)
    if M is None:
        M = torch.empty((B, H, dk, dk), dtype=torch.float32, device=dev)
    _check(M, "M", torch.float32, (B, H, dk, dk), dev)
    with torch.cuda.device(dev):
        st = load_library().kda_chunk_transition(_ptr(q), _ptr(k), _ptr(g), _ptr(beta), _ptr(M),
                                                 B, T, H, dk, _stream(dev))
    if st != KDA_OK:
        raise KdaError("kda_chunk_transition", st)
    return M


def state_chain(M, N, h0=None, *, S_start=None, hT=None):
    """S_0 = h0, S_{p+1} = M_p S_p + N_p over P segments (kda_state_chain).
    M: [B, P, H, dk, dk]; N: [B, P, H, dk, dv]; h0: [B, H, dk, dv] or None.
    Returns (S_start [B, P, H, dk, dv], hT [B, H, dk, dv])."""
    import torch
    B, P, H, dk, dv = N.shape
    dev = _require_cuda(N)
    _check(M, "M", torch.float32, (B, P, H, dk, dk), dev)
    _check(N, "N", torch.float32, (B, P, H, dk, dv), dev)
    if h0 is not None:
        _check(h0, "h0", torch.float32, (B, H, dk, dv), dev)
    if S_start is None:
        S_start = torch.empty_like(N)
    if hT is None:
        hT = torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev)
    _check(S_start, "S_start", torch.float32, (B, P, H, dk, dv), dev)
    _check(hT, "hT", torch.float32, (B, H, dk, dv), dev)
    with torch.cuda.device(dev):
        st = load_library().kda_state_chain(_ptr(M), _ptr(N), _ptr(h0), _ptr(S_start), _ptr(hT),
                                            B, P, H, dk, dv, _stream(dev))
    if st != KDA_OK:
        raise KdaError("kda_state_chain", st)
    return S_start, hT


def chunk_fwd_f32(q, k, v, g, beta, h0=None, *, o=None, hT=None, output_final_state=True):
    """KDA prefill with fp32 inputs/outputs and fp32 arithmetic."""
    import torch
    return _prefill("kda_chunk_fwd_f32", torch.float32, q, k, v, g, beta, h0, o,
                    hT, output_final_state)


def _decode(fn_name, q, k, v, g, beta, state, o):
    import torch
    N, H, dk = q.shape
    dv = v.shape[-1]
    dev = _require_cuda(q)
    for name, t, shp in (("q", q, (N, H, dk)), ("k", k, (N, H, dk)),
                         ("g", g, (N, H, dk)), ("v", v, (N, H, dv)),
                         ("beta", beta, (N, H))):
        _check(t, name, torch.bfloat16, shp, dev)
    _check(state, "state", torch.float32, (N, H, dk, dv), dev)
    if o is None:
        o = torch.empty((N, H, dv), dtype=torch.bfloat16, device=dev)
    _check(o, "o", torch.bfloat16, (N, H, dv), dev)
    with torch.cuda.device(dev):
        st = getattr(load_library(), fn_name)(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                            _ptr(state), _ptr(o), N, H, dk, dv, _stream(dev))
    if st != KDA_OK:
        raise KdaError(fn_name, st)
    return o


def decode_step(q, k, v, g, beta, state, *, o=None):
    """One decode token per request; `state` [N, H, dk, dv] fp32 is updated
    in place.  q, k, g: [N, H, dk]; v: [N, H, dv]; beta: [N, H] (bf16).
    Returns o [N, H, dv] bf16."""
    return _decode("kda_decode_step", q, k, v, g, beta, state, o)


def decode_step_raw(q_raw, k_raw, v, z, beta, state, *, o=None):
    """decode_step with the prologue fused in (kda_decode_step_raw): q_raw,
    k_raw unnormalised, z the gate pre-activation."""
    return _decode("kda_decode_step_raw", q_raw, k_raw, v, z, beta, state, o)




VERIFY_MAX_TOKENS = 64


def verify_fwd(q, k, v, g, beta, h0=None, *, o=None, states=None):
    """K tokens per request from the start states h0, keeping the state after
    every token (kda_verify_fwd).  q, k, g: [N, K, H, dk]; v: [N, K, H, dv];
    beta: [N, K, H] (bf16); h0: [N, H, dk, dv] fp32 or None (read only).
    Returns (o [N, K, H, dv] bf16, states [N, K, H, dk, dv] fp32), with
    states[n, t] the state of request n after its token t + 1."""
    import torch
    N, K, H, dk = q.shape
    dv = v.shape[-1]
    dev = _require_cuda(q)
    for name, t, shp in (("q", q, (N, K, H, dk)), ("k", k, (N, K, H, dk)),
                         ("g", g, (N, K, H, dk)), ("v", v, (N, K, H, dv)),
                         ("beta", beta, (N, K, H))):
        _check(t, name, torch.bfloat16, shp, dev)
    if h0 is not None:
        _check(h0, "h0", torch.float32, (N, H, dk, dv), dev)
    if o is None:
        o = torch.empty((N, K, H, dv), dtype=torch.bfloat16, device=dev)
    if states is None:
        states = torch.empty((N, K, H, dk, dv), dtype=torch.float32, device=dev)
    _check(o, "o", torch.bfloat16, (N, K, H, dv), dev)
    _check(states, "states", torch.float32, (N, K, H, dk, dv), dev)
    with torch.cuda.device(dev):
        st = load_library().kda_verify_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                           _ptr(h0), _ptr(o), _ptr(states), N, K, H, dk, dv,
                                           _stream(dev))
    if st != KDA_OK:
        raise KdaError("kda_verify_fwd", st)
    return o, states


def _bwd(fn_name, q, k, v, g, beta, h0, dO, dhT, want_dh0):
    import torch
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dev = _require_cuda(q)
    for name, t, shp in (("q", q, (B, T, H, dk)), ("k", k, (B, T, H, dk)),
                         ("g", g, (B, T, H, dk)), ("v", v, (B, T, H, dv)),
                         ("beta", beta, (B, T, H)), ("dO", dO, (B, T, H, dv))):
        _check(t, name, torch.bfloat16, shp, dev)
    for name, t in (("h0", h0), ("dhT", dhT)):
        if t is not None:
            _check(t, name, torch.float32, (B, H, dk, dv), dev)
    gq, gk, gg = (torch.empty((B, T, H, dk), dtype=torch.bfloat16, device=dev) for _ in range(3))
    gv = torch.empty((B, T, H, dv), dtype=torch.bfloat16, device=dev)
    gb = torch.empty((B, T, H), dtype=torch.bfloat16, device=dev)
    gh = torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev) if want_dh0 else None
    with torch.cuda.device(dev):
        st = getattr(load_library(), fn_name)(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0),
                                              _ptr(dO), _ptr(dhT), _ptr(gq), _ptr(gk), _ptr(gv), _ptr(gg),
                                              _ptr(gb), _ptr(gh), B, T, H, dk, dv, _stream(dev))
    if st != KDA_OK:
        raise KdaError(fn_name, st)
    return gq, gk, gv, gg, gb, gh


def chunk_bwd(q, k, v, g, beta, h0, dO, dhT=None, *, want_dh0=True):
    """Gradients of chunk_fwd (kda_chunk_bwd): with L = sum(dO * o) +
    sum(dhT * hT), returns (dq, dk, dv, dg, dbeta, dh0); dq, dk, dg, dv,
    dbeta bf16 in the input layouts, dh0 [B, H, dk, dv] fp32 (None if
    want_dh0 is False).  dO: [B, T, H, dv] bf16; dhT: [B, H, dk, dv] fp32 or
    None; h0 as for chunk_fwd."""
    return _bwd("kda_chunk_bwd", q, k, v, g, beta, h0, dO, dhT, want_dh0)


def chunk_bwd_raw(q_raw, k_raw, v, z, beta, h0, dO, dhT=None, *, want_dh0=True):
    """Gradients of chunk_fwd_raw (kda_chunk_bwd_raw): (dq_raw, dk_raw, dv,
    dz, dbeta, dh0), the prologue and its chain rule inside the kernels."""
    return _bwd("kda_chunk_bwd_raw", q_raw, k_raw, v, z, beta, h0, dO, dhT, want_dh0)


# ------------------------------------- one decay per head (gated delta rule) --
GATE_F32_BETA_BF16 = 2

# These calls are made once per layer and token, so their checks are written to
# cost little: one comparison of type, shape and device per tensor, the reason
# looked for only when it fails.

_BF16 = _F32 = _I32 = _torch = None


def _types():
    """torch, with the dtypes the calls compare against at hand."""
    global _BF16, _F32, _I32, _torch
    if _torch is None:
        import torch
        _BF16, _F32, _I32, _torch = torch.bfloat16, torch.float32, torch.int32, torch
    return _torch


def _call(fn_name, dev, *args):
    """The library function on the current stream of `dev`, made the current device."""
    fn = getattr(_lib or load_library(), fn_name)
    # the bindings below torch.cuda.current_device and current_stream: short calls are bound by the host, and those
    # two are 2 to 3 us of a call of 15
    cuda = _torch._C
    if cuda._cuda_getDevice() == dev.index:
        st = fn(*args, cuda._cuda_getCurrentRawStream(dev.index))
    else:
        with _torch.cuda.device(dev):
            st = fn(*args, cuda._cuda_getCurrentRawStream(dev.index))
    if st != KDA_OK:
        raise KdaError(fn_name, st)


def _dense(t, name, dtype, shape, dev):
    """Address of a contiguous tensor of this type and shape (None: None)."""
    if t.dtype is not dtype or t.shape != shape or t.device != dev or not t.is_contiguous():
        _check(t, name, dtype, shape, dev)
    return t.data_ptr()


def _check_tokens(t, name, lead, heads, d, dev):
    """A bf16 tensor [*lead, heads, d] whose heads are dense and whose tokens
    are a constant number of elements apart; returns that number."""
    if t.dtype is not _BF16:
        raise TypeError("%s must be %s, got %s" % (name, _BF16, t.dtype))
    if t.shape != (*lead, heads, d):
        raise ValueError("%s must have shape %s, got %s" % (name, (*lead, heads, d), tuple(t.shape)))
    if t.device != dev:
        raise ValueError("%s must be on %s, got %s" % (name, dev, t.device))
    if t.is_contiguous():
        return heads * d
    st = t.stride()
    if t.numel() == 0:
        return heads * d
    if (d > 1 and st[-1] != 1) or (heads > 1 and st[-2] != d):
        raise ValueError("%s: a token's heads must be dense, got strides %s" % (name, st))
    step, n = None, 1                                # from the last token axis with more than one entry
    for size, s in zip(t.shape[-3::-1], st[-3::-1]):
        if size > 1:
            if step is None:
                step = s
            elif s != step * n:
                raise ValueError("%s: the tokens must be equally spaced, got strides %s" % (name, st))
            n *= size
    if step is None:
        return heads * d
    if step % 8 != 0 or step < heads * d:
        raise ValueError("%s: the token stride must be a multiple of 8 and at least %d, got %d" % (name, heads * d, step))
    return step


def _check_gates(g, beta, shape, dev):
    """Addresses of g and beta and the C calls' gate_f32: both bf16, both fp32, or g fp32 and beta bf16."""
    kind, other = g.dtype, beta.dtype
    if kind is not _F32 and kind is not _BF16:
        raise TypeError("g must be torch.float32 or torch.bfloat16, got %s" % kind)
    if other is not kind and (kind is _BF16 or other is not _BF16):
        raise TypeError("beta must be %s%s, got %s" % (kind, " or torch.bfloat16" if kind is _F32 else "", other))
    return (_dense(g, "g", kind, shape, dev), _dense(beta, "beta", other, shape, dev),
            0 if kind is _BF16 else 1 if other is _F32 else GATE_F32_BETA_BF16)


def _gdn_sequences(B, T, cu_seqlens, dev):
    """(N, T of the C call) with or without cu_seqlens."""
    if cu_seqlens is None:
        return B, T
    if B != 1:
        raise ValueError("with cu_seqlens the tokens are packed: the first axis must be 1, got %d" % B)
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must have shape (N + 1,), got %s" % (tuple(cu_seqlens.shape),))
    _dense(cu_seqlens, "cu_seqlens", _I32, cu_seqlens.shape, dev)
    return cu_seqlens.shape[0] - 1, T


def gdn_chunk_fwd(q, k, v, g, beta, h0=None, *, scale=1.0, cu_seqlens=None, slots=None, o=None, hT=None,
                  output_final_state=True):
    """Chunked forward of the gated delta rule with one decay per head
    (kda_gdn_chunk_fwd), bf16 in and out, fp32 state.

    q, k: [B, T, HK, 128]; v: [B, T, HV, 128] (bf16; slices of one wider tensor
    are taken as they are); g, beta: [B, T, HV], fp32 or bf16, or an fp32 g with
    a bf16 beta.  With cu_seqlens (int32 [N + 1], not decreasing, on the device)
    B is 1 and sequence n has the tokens [cu_seqlens[n], cu_seqlens[n + 1]); else
    N = B.

    h0: [N, HV, 128, 128] fp32 or None; hT may be passed as h0.  With slots
    (int32 [N], on the device) h0 is a pool [rows, HV, 128, 128]: sequence n
    starts from row slots[n] and its last state is written there; a slot
    outside the pool starts from zero and keeps none.  Rows of o that belong to
    no sequence are not written.  Returns (o, hT), hT the pool with slots."""
    _types()
    B, T, HK, dk = q.shape
    HV, dv = v.shape[-2:]
    dev = _require_cuda(q)
    qs = _check_tokens(q, "q", (B, T), HK, dk, dev)
    ks = _check_tokens(k, "k", (B, T), HK, dk, dev)
    vs = _check_tokens(v, "v", (B, T), HV, dv, dev)
    gp, bp, gf = _check_gates(g, beta, (B, T, HV), dev)
    N, Tc = _gdn_sequences(B, T, cu_seqlens, dev)
    rows, sp = N, None
    if slots is not None:
        if h0 is None:
            raise ValueError("slots name rows of a pool of states: h0 must be given")
        if hT is not None and hT is not h0:
            raise ValueError("with slots the last states are written to the pool: hT must not be another tensor")
        sp = _dense(slots, "slots", _I32, (N,), dev)
        rows = h0.shape[0]
        hT = h0 if output_final_state else None
    state = (rows, HV, dk, dv)
    hp = None if h0 is None else _dense(h0, "h0", _F32, state, dev)
    if o is None:
        o = v.new_empty((B, T, HV, dv))
    if hT is None and output_final_state:
        hT = v.new_empty(state, dtype=_F32)
    _call("kda_gdn_chunk_fwd", dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), gp, bp, hp,
          _dense(o, "o", _BF16, (B, T, HV, dv), dev), None if hT is None else _dense(hT, "hT", _F32, state, dev),
          None if cu_seqlens is None else cu_seqlens.data_ptr(), sp, rows, scale, N, Tc, HK, HV, dk, dv, qs, ks, vs, gf)
    return o, hT


def gdn_chunk_bwd(q, k, v, g, beta, h0, dO, dhT=None, *, scale=1.0, cu_seqlens=None, want_dh0=True):
    """Gradients of gdn_chunk_fwd (kda_gdn_chunk_bwd): with L = sum(dO * o) +
    sum(dhT * hT), returns (dq, dk, dv, dg, dbeta, dh0).

    q, k and v are bf16 as in the forward, or all three a Packed8 (their
    8-bit checkpoints; the gradients are those at the values that these stand
    for).  dO: [B, T, HV, 128] bf16; dhT: [N, HV, 128, 128] fp32 or None.  dq,
    dk (summed over the value heads of a group), dv, dg, dbeta are bf16, dh0 is
    fp32 (None if want_dh0 is False).  Tokens that belong to no sequence get
    zero gradients."""
    _types()
    eight = isinstance(q, Packed8)
    if isinstance(k, Packed8) != eight or isinstance(v, Packed8) != eight:
        raise TypeError("q, k and v must all be tensors or all be Packed8")
    B, T, HK, dk = q.shape
    HV, dv = v.shape[-2:]
    dev = _require_cuda(q.data if eight else q)
    if eight:
        ins, scales, strides = zip(*((*_packed8(t, name, (B, T, heads, d), dev), heads * d) for name, t, heads, d in
                                     (("q", q, HK, dk), ("k", k, HK, dk), ("v", v, HV, dv))))
    else:
        strides = (_check_tokens(q, "q", (B, T), HK, dk, dev), _check_tokens(k, "k", (B, T), HK, dk, dev),
                   _check_tokens(v, "v", (B, T), HV, dv, dev))
        ins = (q.data_ptr(), k.data_ptr(), v.data_ptr())
    gp, bp, gf = _check_gates(g, beta, (B, T, HV), dev)
    N, Tc = _gdn_sequences(B, T, cu_seqlens, dev)
    state = (N, HV, dk, dv)
    gq, gk, gv, gg, gb = (dO.new_empty(shape, dtype=_BF16) for shape in
                          ((B, T, HK, dk), (B, T, HK, dk), (B, T, HV, dv), (B, T, HV), (B, T, HV)))
    gh = dO.new_empty(state, dtype=_F32) if want_dh0 else None
    rest = (gp, bp, None if h0 is None else _dense(h0, "h0", _F32, state, dev), _dense(dO, "dO", _BF16, (B, T, HV, dv), dev),
            None if dhT is None else _dense(dhT, "dhT", _F32, state, dev), gq.data_ptr(), gk.data_ptr(), gv.data_ptr(),
            gg.data_ptr(), gb.data_ptr(), None if gh is None else gh.data_ptr(),
            None if cu_seqlens is None else cu_seqlens.data_ptr(), scale, N, Tc, HK, HV, dk, dv)
    if eight:
        _call("kda_gdn_chunk_bwd_packed8", dev, *ins, *scales, *rest, gf)
    else:
        _call("kda_gdn_chunk_bwd", dev, *ins, *rest, *strides, gf)
    return gq, gk, gv, gg, gb, gh


def gdn_decode_step(q, k, v, g, beta, state, *, scale=1.0, slots=None, o=None):
    """One token per request of the gated delta rule with one decay per head
    (kda_gdn_decode_step); `state` is updated in place.

    q, k: [N, HK, dk]; v: [N, HV, dv] (bf16; slices of one wider tensor are
    taken as they are); g, beta: [N, HV], fp32 or bf16, or an fp32 g with a bf16
    beta; state: fp32
    [N, HV, dk, dv], or a pool [rows, HV, dk, dv] with slots [N] (int32, on the
    device) naming each request's row; a slot outside the pool marks a padded
    request (o = 0, no state).  Returns o [N, HV, dv] bf16."""
    _types()
    N, HK, dk = q.shape
    HV, dv = v.shape[-2:]
    dev = _require_cuda(q)
    qs = _check_tokens(q, "q", (N,), HK, dk, dev)
    ks = _check_tokens(k, "k", (N,), HK, dk, dev)
    vs = _check_tokens(v, "v", (N,), HV, dv, dev)
    gp, bp, gf = _check_gates(g, beta, (N, HV), dev)
    rows, sp = (N, None) if slots is None else (state.shape[0], _dense(slots, "slots", _I32, (N,), dev))
    if o is None:
        o = v.new_empty((N, HV, dv))
    _call("kda_gdn_decode_step", dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), gp, bp,
          _dense(state, "state", _F32, (rows, HV, dk, dv), dev), _dense(o, "o", _BF16, (N, HV, dv), dev), sp, rows,
          scale, N, HK, HV, dk, dv, qs, ks, vs, gf)
    return o


# ------------------------------------------- activation checkpoints in 8 bits --

class Packed8(NamedTuple):
    """A bf16 tensor's 8-bit form: data (torch.float8_e4m3fn, the tensor's
    shape) and scales (uint8, one per 32 channels of the last axis, the biased
    exponent of a power of two)."""
    data: "torch.Tensor"
    scales: "torch.Tensor"

    @property
    def shape(self):
        return self.data.shape


ACT8_MAX_TENSORS = 4
_PTRS = [ctypes.c_void_p * n for n in range(ACT8_MAX_TENSORS + 1)]
_SIZES = [ctypes.c_int64 * n for n in range(ACT8_MAX_TENSORS + 1)]


def _act8_rows(t, name, dev):
    """(rows, channels of a row, elements from row to row) of a bf16 tensor; the
    last two axes make one row where they are dense."""
    shape = t.shape
    if len(shape) < 1 or shape[-1] % 32 != 0:
        raise ValueError("%s: the last axis must be a multiple of 32, got shape %s" % (name, tuple(shape)))
    if len(shape) < 3 or (shape[-2] > 1 and t.stride(-2) != shape[-1]):
        t = t.unsqueeze(-2)
    heads, d = t.shape[-2:]
    stride = _check_tokens(t, name, t.shape[:-2], heads, d, dev)
    return t.numel() // (heads * d) if heads * d else 0, heads * d, stride


def act_pack8(*tensors):
    """The 8-bit form (Packed8) of each of up to four bf16 tensors, in one
    launch (kda_act_pack8).  The last axis must be a multiple of 32; the
    tensors may be slices of wider ones as long as their rows (all axes but the
    last, or but the last two where these are dense) are equally spaced, a
    multiple of 8 elements apart.  One tensor gives a Packed8, several a tuple of them."""
    torch = _types()
    n = len(tensors)
    if not 1 <= n <= ACT8_MAX_TENSORS:
        raise ValueError("act_pack8 takes 1 to %d tensors, got %d" % (ACT8_MAX_TENSORS, n))
    dev = _require_cuda(tensors[0])
    rows, cols, strides, out = [], [], [], []
    for i, t in enumerate(tensors):
        shape = t.shape
        r, c, stride = _act8_rows(t, "tensor %d" % i, dev)
        rows.append(r)
        cols.append(c)
        strides.append(stride)
        out.append(Packed8(t.new_empty(shape, dtype=torch.float8_e4m3fn),
                           t.new_empty((*shape[:-1], shape[-1] // 32), dtype=torch.uint8)))
    _call("kda_act_pack8", dev, n, _PTRS[n](*[t.data_ptr() for t in tensors]), _PTRS[n](*[p.data.data_ptr() for p in out]),
          _PTRS[n](*[p.scales.data_ptr() for p in out]), _SIZES[n](*rows), _SIZES[n](*cols), _SIZES[n](*strides))
    return out[0] if n == 1 else tuple(out)


def _packed8(p, name, shape, dev):
    """Addresses of a Packed8's data and scales, checked against the tensor's shape."""
    if len(shape) < 1 or shape[-1] % 32 != 0:
        raise ValueError("%s: the last axis must be a multiple of 32, got shape %s" % (name, tuple(shape)))
    return (_dense(p.data, name + ".data", _torch.float8_e4m3fn, shape, dev),
            _dense(p.scales, name + ".scales", _torch.uint8, (*shape[:-1], shape[-1] // 32), dev))


def act_unpack8(packed, *, out=None):
    """The bf16 values that a Packed8 stands for, exactly (kda_act_unpack8)."""
    _types()
    dev = _require_cuda(packed.data)
    shape = packed.data.shape
    data, scales = _packed8(packed, "packed", shape, dev)
    if out is None:
        out = packed.data.new_empty(shape, dtype=_BF16)
    last = shape[-1]
    _call("kda_act_unpack8", dev, 1, _PTRS[1](data), _PTRS[1](scales), _PTRS[1](_dense(out, "out", _BF16, shape, dev)),
          _SIZES[1](packed.data.numel() // last if last else 0), _SIZES[1](last))
    return out
