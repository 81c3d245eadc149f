"""Rotary positions with several axes against complex rotations in float64:
layouts, sections that are no multiple of a vector, far and negative positions,
strides, in place, another stream; and the refusals, without a GPU."""

import ctypes
import math
import os

import numpy as np
import pytest
import torch

import attention_distillation_kl_gb300 as skl

A = 4096  # a 16-byte aligned fake address: never dereferenced, validation fails first
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(skl.library_path):
        import __graft_entry__
        __graft_entry__.build()
    return skl.lib()


def rotary(**kw):
    f = dict(positions=A, stride_axis=256, stride_b=128, inv_freq=A, axes=2, section=(16, 16), interleaved=0)
    f.update(kw)
    sec = tuple(f["section"]) + (0,) * (4 - len(f["section"]))
    return skl._Rotary(f["positions"], f["stride_axis"], f["stride_b"], f["inv_freq"], f["axes"],
                       (ctypes.c_int * 4)(*sec), f["interleaved"])


def call(L, x=None, y=None, r=None, B=2, H=2, N=128, d=64, inverse=0):
    v = skl._View(A, H * N * d, N * d, d)
    return L.streamkl_rotate(x or v, y or skl._View(2 * A, H * N * d, N * d, d), r or rotary(), B, H, N, d, inverse, None)


@pytest.mark.parametrize("kw,status", [
    (dict(r=rotary(axes=0)), skl.STREAMKL_INVALID_ARG), (dict(r=rotary(axes=5)), skl.STREAMKL_INVALID_ARG),
    (dict(r=rotary(section=(16, 0))), skl.STREAMKL_INVALID_ARG),
    (dict(r=rotary(section=(16, 17))), skl.STREAMKL_INVALID_ARG),       # 66 of 64 values
    (dict(r=rotary(section=(2 ** 31 - 1, 16))), skl.STREAMKL_INVALID_ARG),
    (dict(r=rotary(interleaved=2)), skl.STREAMKL_INVALID_ARG), (dict(inverse=2), skl.STREAMKL_INVALID_ARG),
    (dict(r=rotary(positions=0)), skl.STREAMKL_INVALID_ARG), (dict(r=rotary(inv_freq=A + 2)), skl.STREAMKL_INVALID_ARG),
    (dict(r=rotary(stride_b=-1)), skl.STREAMKL_INVALID_ARG),
    (dict(d=24), skl.STREAMKL_UNSUPPORTED), (dict(d=272), skl.STREAMKL_UNSUPPORTED),
    (dict(x=skl._View(A + 8, 64, 64, 64)), skl.STREAMKL_INVALID_ARG),
    (dict(y=skl._View(A, 64, 64, 60)), skl.STREAMKL_INVALID_ARG),
    (dict(y=skl._View(A, 2 * 128 * 128, 128 * 128, 128)), skl.STREAMKL_INVALID_ARG),  # x's memory in another order
    (dict(B=-1), skl.STREAMKL_INVALID_ARG), (dict(B=40000), skl.STREAMKL_INVALID_ARG),
])
def test_refusals(L, kw, status):
    assert call(L, **kw) == status


def test_empty_is_no_op(L):
    none = skl._View(0, 0, 0, 0)
    assert call(L, x=none, y=none, N=0) == skl.STREAMKL_OK


def test_binding_refuses_without_a_gpu():
    with pytest.raises(TypeError):
        skl.Rotary(torch.ones(4), torch.zeros((1, 3), dtype=torch.int32))
    with pytest.raises(TypeError):
        skl.streamkl_rotate(torch.zeros((1, 1, 3, 16), dtype=torch.bfloat16), None)


def reference(x, pos, freq, sections, interleaved, inverse):
    """Float64, and the size of each value's pair."""
    x, freq = x.float().cpu().double().numpy(), freq.cpu().double().numpy()
    pos = pos.cpu().numpy().astype(np.float64)
    if pos.ndim == 2:
        pos = np.repeat(pos[:, None], x.shape[0], 1)
    R = len(freq)
    axis = np.repeat(np.arange(len(sections)), sections)
    # whole turns taken off in integers of 2^-64 turns where positions are far: the product itself needs 31 + 24 bits
    angle = np.remainder(pos[axis].transpose(1, 2, 0).astype(np.longdouble) * freq.astype(np.longdouble),
                         2 * np.longdouble(math.pi) if np.finfo(np.longdouble).eps > 1e-18 else
                         np.longdouble("6.283185307179586476925286766559")).astype(np.float64)
    turn = np.exp((-1j if inverse else 1j) * angle)[:, None]
    a, b = (slice(0, 2 * R, 2), slice(1, 2 * R, 2)) if interleaved else (slice(0, R), slice(R, 2 * R))
    z = (x[..., a] + 1j * x[..., b]) * turn
    out, size = x.copy(), np.zeros(x.shape)
    out[..., a], out[..., b] = z.real, z.imag
    size[..., a] = size[..., b] = np.abs(z)
    return out, size


def bound(want, size, far=0.0):
    """One rounding to bf16; angles off by 2^-32 turns (the fraction kept), a
    fp32 rounding of half turns (2^-24 of at most pi) and what the longest
    position times the 53-bit fraction leaves; sincospi and the two products,
    8 fp32 roundings of the pair's size in all."""
    angle = 2 * math.pi * 2.0 ** -32 + math.pi * 2.0 ** -24 + far
    return 2.0 ** -8 * np.abs(want) + size * (angle + 8 * 2.0 ** -24) * (1 + 2.0 ** -8) + 1e-38


def make(B, H, N, d, bshd, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((B, H, N, d), generator=g).to(torch.bfloat16)
    return x.transpose(1, 2).contiguous().cuda().transpose(1, 2) if bshd else x.cuda()


CASES = [
    # B, H, N, d, sections, interleaved, bshd
    (1, 1, 1, 16, [8], False, False),
    (1, 1, 1, 16, [1], True, False),
    (2, 3, 37, 64, [8, 12, 12], False, True),
    (1, 32, 300, 128, [16, 24, 24], False, True),
    (1, 32, 300, 128, [16, 24, 24], True, True),
    (3, 5, 77, 96, [18, 18], True, False),
    (2, 2, 129, 112, [5, 7, 11, 3], False, False),      # 26 pairs: a pair at a time
    (2, 2, 129, 112, [5, 7, 11, 2], True, True),        # 25 pairs
    (1, 7, 1000, 256, [128], False, False),
    (1, 2, 65, 80, [3, 1, 4], False, True),             # 8 pairs, 64 values copied
]


@gpu
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("B,H,N,d,sections,inter,bshd", CASES)
def test_against_complex_rotation(B, H, N, d, sections, inter, bshd, inverse):
    g = torch.Generator().manual_seed(3)
    x = make(B, H, N, d, bshd)
    R = sum(sections)
    freq = (10000.0 ** (-torch.arange(R) / R)).float().cuda()
    pos = torch.randint(-5000, 100000, (len(sections), B, N), generator=g, dtype=torch.int32).cuda()
    rot = skl.Rotary(freq, pos, sections, interleaved=inter)
    y = skl.streamkl_rotate(x, rot, inverse=inverse)
    want, size = reference(x, pos, freq, sections, inter, inverse)
    got = y.float().cpu().double().numpy()
    assert np.all(np.abs(got - want) <= bound(want, size))
    assert torch.equal(y[..., 2 * R:], x[..., 2 * R:])
    z = x.clone(memory_format=torch.preserve_format)
    assert skl.streamkl_rotate(z, rot, inverse=inverse, out=z) is z and torch.equal(z, y)


@gpu
def test_far_positions():
    x = make(1, 2, 64, 64, False)
    freq = (10000.0 ** (-torch.arange(32) / 32)).float().cuda()
    pos = (torch.arange(64, dtype=torch.int64) * 33554431 - 2 ** 30 + 7).to(torch.int32).reshape(1, 64).cuda()
    y = skl.streamkl_rotate(x, skl.Rotary(freq, pos))
    want, size = reference(x, pos, freq, [32], False, False)
    # 2^31 positions of a fraction rounded to 2^-53 of a turn (twice: the factor 1 / 2 pi and the product)
    assert np.all(np.abs(y.float().cpu().double().numpy() - want) <= bound(want, size, 2 * math.pi * 2.0 ** -21))


@gpu
def test_shared_positions_views_and_streams():
    big = make(2, 4, 50, 128, False)
    x = big[:, 1:3, 5:45, 32:96]  # a slice of heads, tokens and values
    freq = (100.0 ** (-torch.arange(32) / 32)).float().cuda()
    pos = torch.arange(80, dtype=torch.int32).reshape(2, 40).cuda()
    one = skl.Rotary(freq, pos, [20, 12])
    y = skl.streamkl_rotate(x, one)
    each = skl.Rotary(freq, pos[:, None].expand(2, 2, 40), [20, 12])
    assert torch.equal(skl.streamkl_rotate(x, each), y)
    want, size = reference(x, pos, freq, [20, 12], False, False)
    assert np.all(np.abs(y.float().cpu().double().numpy() - want) <= bound(want, size))
    out = torch.zeros((2, 50, 2, 96), dtype=torch.bfloat16, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    skl.streamkl_rotate(x, one, out=out[:, 3:43, :, 16:80].transpose(1, 2), stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(out[:, 3:43, :, 16:80].transpose(1, 2), y)
    out[:, 3:43, :, 16:80] = 0
    assert not out.any()


@gpu
def test_inverse_is_the_gradient():
    """<R x, g> = <x, R^-1 g>, and R^-1 R x = x, up to the roundings of each."""
    x, g = make(2, 3, 90, 64, True, 1), make(2, 3, 90, 64, False, 2)
    freq = (1000.0 ** (-torch.arange(20) / 20)).float().cuda()
    pos = torch.arange(3 * 2 * 90, dtype=torch.int32).reshape(3, 2, 90).cuda()
    rot = skl.Rotary(freq, pos, [7, 7, 6], interleaved=True)
    a = (skl.streamkl_rotate(x, rot).double() * g.double())
    b = (skl.streamkl_rotate(g, rot, inverse=True).double() * x.double())
    size = (x.double().norm() * g.double().norm())
    assert abs(a.sum() - b.sum()) <= 2 * (2.0 ** -8 + 2.0 ** -20) * size
    back = skl.streamkl_rotate(skl.streamkl_rotate(x, rot), rot, inverse=True).double()
    assert (back - x.double()).norm() <= (2 * 2.0 ** -8 + 2.0 ** -14) * x.double().norm()


@gpu
def test_binding_refusals():
    x = make(1, 2, 8, 32, False)
    freq, pos = torch.ones(16, device="cuda"), torch.zeros((1, 8), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        skl.Rotary(freq, pos, [8, 8])
    with pytest.raises(TypeError):
        skl.Rotary(freq, pos.long())
    with pytest.raises(ValueError):
        skl.streamkl_rotate(x, skl.Rotary(freq, pos[:, :7]))
    with pytest.raises(skl.StreamKLError):
        skl.streamkl_rotate(x, skl.Rotary(torch.ones(17, device="cuda"), pos))  # 34 of 32 values
    with pytest.raises(ValueError):
        skl.streamkl_rotate(x, skl.Rotary(freq, pos), out=x.float())
