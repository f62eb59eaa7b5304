"""Activation checkpoints in 8 bits (kda_act_pack8, kda_act_unpack8): equal,
bit for bit, to the definition in 64 bits.  No tolerance: the scale is read off
the largest magnitude's bits and the one rounding is to the nearest e4m3, ties
to even."""
import ctypes

import numpy as np
import pytest
import torch

import linear_attention_07_b200 as kda


def definition(x):
    """(scales, values) of a bf16 tensor, fp64 arithmetic on the host."""
    y = x.detach().cpu().double().unflatten(-1, (-1, 32)).numpy()
    top = np.abs(y).max(-1, keepdims=True)
    m, e = np.frexp(top)                             # top = m 2^e, m in [1/2, 1); 448 = 0.875 * 2^9
    e = np.where(m <= 0.875, e - 9, e - 8)
    e = np.where(top > 0, np.maximum(e, -127), -127)
    z = y / np.exp2(e)
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(z), 2.0 ** -20))), -6) - 3)
    z = np.rint(z / step) * step                     # rint: ties to even
    z = np.where(e == 120, np.clip(z, -240, 240), z)  # 256 * 2^120 is past bf16's largest number
    return (e + 127).astype(np.uint8)[..., 0], (z * np.exp2(e)).reshape(x.shape)


def check(x, p):
    s, v = definition(x)
    assert np.array_equal(p.scales.cpu().numpy(), s)
    back = kda.act_unpack8(p)
    assert back.dtype == torch.bfloat16 and back.shape == x.shape
    assert np.array_equal(back.double().cpu().numpy(), v)


def test_refusals():
    lib = kda.load_library()
    n0 = lib.kda_launch_count()
    P, I = ctypes.c_void_p, ctypes.c_int64
    ok = dict(count=1, x=0x10000, d=0x20000, s=0x30001, rows=2, cols=64, stride=64)

    def pack(**kw):
        a = dict(ok, **kw)
        return lib.kda_act_pack8(a["count"], (P * 1)(a["x"]), (P * 1)(a["d"]), (P * 1)(a["s"]), (I * 1)(a["rows"]),
                                 (I * 1)(a["cols"]), (I * 1)(a["stride"]), None)

    for bad in (dict(count=0), dict(count=5), dict(x=0), dict(x=0x10008), dict(d=0x20004), dict(s=0), dict(rows=-1),
                dict(cols=48), dict(cols=-32), dict(stride=60), dict(stride=56), dict(stride=68)):
        assert pack(**bad) == kda.KDA_ERR_INVALID_ARG, bad
    assert pack(rows=1 << 41) == kda.KDA_ERR_UNSUPPORTED
    assert pack(rows=0, x=0) == kda.KDA_OK
    assert lib.kda_act_unpack8(1, (P * 1)(0x10000), (P * 1)(0), (P * 1)(0x20000), (I * 1)(2), (I * 1)(64), None) == kda.KDA_ERR_INVALID_ARG
    assert lib.kda_act_pack8(1, None, None, None, None, None, None, None) == kda.KDA_ERR_INVALID_ARG
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        kda.act_pack8(x)
    with pytest.raises(ValueError):
        kda.act_pack8()
    with pytest.raises(ValueError, match="CUDA"):
        kda.act_unpack8(kda.Packed8(torch.zeros(4, 64, dtype=torch.float8_e4m3fn), torch.zeros(4, 2, dtype=torch.uint8)))
    assert lib.kda_launch_count() == n0


def test_sizes_past_64_bits_are_refused():
    """rows * cols past 2^63: neither taken for nothing to do nor for few rows."""
    lib = kda.load_library()
    n0 = lib.kda_launch_count()
    P, I = ctypes.c_void_p, ctypes.c_int64
    for rows, cols in ((1 << 39, 1 << 30), (1 << 38, 1 << 30), ((1 << 38) + 1, 1 << 30), ((1 << 40) - 1, (1 << 31) - 32), (1 << 35, 1 << 10)):
        args = (1, (P * 1)(0x10000), (P * 1)(0x20000), (P * 1)(0x30000), (I * 1)(rows), (I * 1)(cols))
        assert lib.kda_act_pack8(*args, (I * 1)(cols), None) == kda.KDA_ERR_UNSUPPORTED, (rows, cols)
        assert lib.kda_act_unpack8(*args, None) == kda.KDA_ERR_UNSUPPORTED, (rows, cols)
    assert lib.kda_launch_count() == n0


ROWS = [((2, 50, 1024), (slice(None), slice(None), slice(0, 256)), (100, 256, 1024)),      # [B, T, d] of a projection
        ((2, 50, 8, 128), (slice(None), slice(None), slice(2, 6)), (100, 512, 1024)),       # whole heads
        ((2, 50, 8, 128), (slice(None), slice(None), slice(None), slice(0, 64)), (800, 64, 128)),   # part of every head
        ((50, 1024), (slice(None), slice(256, 512)), (50, 256, 1024)),
        ((4, 50, 1024), (slice(None, None, 2), slice(0, 1), slice(0, 32)), (2, 32, 102400)),
        ((3, 4, 64), (slice(None),), (3, 256, 256)), ((96,), (slice(32, 64),), (1, 32, 32)), ((0, 4, 128), (slice(None),), (0, 512, 512))]


@pytest.mark.parametrize("shape, part, want", ROWS, ids=str)
def test_rows_of_slices(shape, part, want):
    """(rows, channels, stride) of a slice: the last axis is split from the ones before it wherever these are equally spaced."""
    kda._types()
    x = torch.zeros(shape, dtype=torch.bfloat16)[part]
    assert kda._act8_rows(x, "x", x.device) == want


def test_rows_that_are_refused():
    kda._types()
    wide = torch.zeros(2, 50, 8, 128, dtype=torch.bfloat16)
    for bad in (wide[:, :40, :, :64], wide[..., ::2], wide[:, ::3],
                wide[:1, :1, :1].expand(1, 5, 1, 128), wide[0, 0, 0, :64].expand(3, 64), wide.transpose(1, 2)):
        with pytest.raises(ValueError):
            kda._act8_rows(bad, "x", bad.device)
    with pytest.raises(ValueError, match="32"):
        kda._act8_rows(wide[..., :48], "x", wide.device)
    with pytest.raises(TypeError):
        kda._act8_rows(wide.float(), "x", wide.device)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(32,), (1, 32), (3, 96), (7, 5, 64), (2, 77, 3, 128), (1000, 1, 128), (0, 4, 128)], ids=str)
def test_shapes(shape):
    x = torch.randn(shape, device="cuda").to(torch.bfloat16)
    check(x, kda.act_pack8(x))


@pytest.mark.gpu
def test_slices_in_one_launch():
    """q, k, v of one projection, as they are, in one launch."""
    qkv = torch.randn(2, 50, 2 * 256 + 512, device="cuda").to(torch.bfloat16)
    q, k, v = (t.unflatten(-1, (-1, 128)) for t in qkv.split([256, 256, 512], dim=-1))
    n0 = kda.launch_count()
    packed = kda.act_pack8(q, k, v)
    assert kda.launch_count() == n0 + 1
    for x, p in zip((q, k, v), packed):
        check(x, p)
    check(qkv[0, :, :256], kda.act_pack8(qkv[0, :, :256]))


@pytest.mark.gpu
def test_every_magnitude():
    """Every finite bf16 value as a block's largest, ties and subnormals among them."""
    bits = torch.arange(0, 0x7f80, dtype=torch.int32).to(torch.int16)
    top = bits.view(torch.bfloat16).cuda()
    x = top[:, None].float() * torch.linspace(-1, 1, 32, device="cuda")
    x = x.to(torch.bfloat16)
    x[:, 7] = top
    check(x, kda.act_pack8(x))


@pytest.mark.gpu
def test_ties_go_to_even():
    """All halves between neighbours of e4m3 at one scale."""
    grid = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    mid = ((grid[1:] + grid[:-1]) / 2)
    x = torch.zeros(len(mid), 32, dtype=torch.float64)
    x[:, 0], x[:, 1], x[:, 2] = 448.0, mid, -mid
    assert bool((x.to(torch.bfloat16).double() == x).all())
    x = x.to(torch.bfloat16).cuda()
    check(x, kda.act_pack8(x))


@pytest.mark.gpu
def test_not_numbers():
    """A block with a NaN or an infinity reads as NaN; its neighbours stay."""
    x = torch.randn(3, 96, device="cuda").to(torch.bfloat16)
    x[0, 40], x[1, 0], x[2, 95] = float("nan"), float("inf"), -float("inf")
    p = kda.act_pack8(x)
    back = kda.act_unpack8(p)
    bad = torch.zeros(3, 3, dtype=torch.bool)
    bad[0, 1] = bad[1, 0] = bad[2, 2] = True
    assert bool((p.scales.cpu() == 255).eq(bad).all())
    assert bool(torch.isnan(back).unflatten(-1, (3, 32)).all(-1).cpu().eq(bad).all())
    good = ~bad
    _, v = definition(torch.where(torch.isfinite(x), x, 0))
    assert np.array_equal(back.double().cpu().unflatten(-1, (3, 32))[good].numpy(), torch.from_numpy(v).unflatten(-1, (3, 32))[good].numpy())


@pytest.mark.gpu
def test_refusals_of_the_binding():
    x = torch.randn(4, 64, device="cuda")
    with pytest.raises(TypeError):
        kda.act_pack8(x)
    with pytest.raises(ValueError):
        kda.act_pack8(x.to(torch.bfloat16)[:, :48])
    with pytest.raises(ValueError):
        kda.act_pack8(x.to(torch.bfloat16)[:, ::2])
    with pytest.raises(TypeError):
        kda.act_unpack8(kda.Packed8(x.to(torch.bfloat16), torch.zeros(4, 2, dtype=torch.uint8, device="cuda")))


@pytest.mark.gpu
@pytest.mark.parametrize("shape, part, rows", ROWS, ids=str)
def test_slices(shape, part, rows):
    x = torch.randn(shape, device="cuda").to(torch.bfloat16)[part]
    check(x, kda.act_pack8(x))
