"""Rotary positions: plan and refusals on the CPU, parity with the float64
oracle on the GPU.

Tolerance: the angle's fraction of a turn is exact to 2^-32, its fp32 value
and the sine and cosine are each off by at most a few 2^-24, so an fp32
result is within 8 * 2^-24 of |u| + |v| (two products, a sum, the sine, the
cosine and their amplitude); a bf16 result is that rounded once, by at most
2^-8 of its value.
"""
import numpy as np
import pytest
import torch

import exact_tiled_softmax_attn_gb300 as B
from oracle import scored as ref

from parity import np64


def test_plan_frequencies():
    for kw in (dict(rot=128), dict(rot=64, theta=500000.0, factor=8.0), dict(rot=2, theta=2.0),
               dict(rot=256, factor=16.0, original_length=8192.0, low_turns=1.0, high_turns=32.0)):
        p = B.rope_plan(**kw)
        want = ref.rope_frequencies(**kw)
        got = np.array([t / 2.0 ** 64 for t in p.turns[:kw["rot"] // 2]]) * 2 * np.pi
        # rounded to 2^-64 of a turn, after a few double-precision steps
        assert (np.abs(got - want) <= 2 * np.pi * 2.0 ** -64 + 1e-14 * want).all()
        assert not any(p.turns[kw["rot"] // 2:])


@pytest.mark.parametrize("kw", [dict(rot=0), dict(rot=3), dict(rot=258), dict(rot=-2), dict(rot=64, theta=1.0),
                                dict(rot=64, theta=float("nan")), dict(rot=64, factor=0.5),
                                dict(rot=64, original_length=-1.0), dict(rot=64, mscale=0.0),
                                dict(rot=64, mscale=1e-60), dict(rot=64, factor=float("inf")),
                                dict(rot=64, original_length=100.0, low_turns=4.0, high_turns=4.0),
                                dict(rot=64, interleaved=2)])
def test_plan_refusals(kw):
    with pytest.raises(B.AttnError) as e:
        B.rope_plan(**kw)
    assert e.value.status == B.ATTN_ERR_INVALID_ARG


D = [8 * 64, 8 * 64, 64]   # contiguous [1, 8, 8, 64]: batch, head, token


def _rope(**kw):
    a = dict(plan=B.rope_plan(64), Q=0x100000, Qout=0x200000, K=0x300000, Kout=0x400000,
             strides=[4096, 512, 64] * 2 + [2048, 512, 64] * 2, pos=0x500000, B=1, H=8, Hkv=4, T=8, d=64, inverse=0,
             dtype=B.ATTN_BF16, stream=0, check=False)
    a.update(kw)
    return B.attn_rope(**a)


@pytest.mark.parametrize("kw,status", [
    (dict(plan=None), B.ATTN_ERR_INVALID_ARG),
    (dict(B=-1), B.ATTN_ERR_INVALID_ARG),
    (dict(Hkv=-1), B.ATTN_ERR_INVALID_ARG),
    (dict(inverse=2), B.ATTN_ERR_INVALID_ARG),
    (dict(dtype=9), B.ATTN_ERR_INVALID_ARG),
    (dict(d=32), B.ATTN_ERR_INVALID_ARG),                     # rot > d
    (dict(d=264), B.ATTN_ERR_UNSUPPORTED),
    (dict(Q=None), B.ATTN_ERR_INVALID_ARG),
    (dict(K=0x300001), B.ATTN_ERR_MISALIGNED),
    (dict(pos=0x500002), B.ATTN_ERR_MISALIGNED),
    (dict(strides=[-1] + [4096, 512, 64, 4096, 512] + [2048, 512, 64] * 2), B.ATTN_ERR_INVALID_ARG),
    (dict(strides=[4096, 512, 64, 4096, 0, 64] + [2048, 512, 64] * 2), B.ATTN_ERR_INVALID_ARG),   # outputs meet
    (dict(strides=[4096, 512, 64, 4096, 512, 32] + [2048, 512, 64] * 2), B.ATTN_ERR_INVALID_ARG),
    (dict(Qout=0x100080), B.ATTN_ERR_INVALID_ARG),            # partly over its own input
    (dict(Kout=0x200000), B.ATTN_ERR_INVALID_ARG),            # over the other output
    (dict(Qout=0x300000), B.ATTN_ERR_INVALID_ARG),            # over the other input
    (dict(pos=0x200000), B.ATTN_ERR_INVALID_ARG),
    (dict(B=0), B.ATTN_OK),
    (dict(T=0, Q=None), B.ATTN_OK),
    (dict(H=0, Hkv=0), B.ATTN_OK),
])
def test_refusals(kw, status):
    assert _rope(**kw) == status


def test_wrapper_refusals():
    q, k = torch.zeros(1, 4, 8, 64), torch.zeros(1, 2, 8, 64)
    plan = B.rope_plan(64)
    for a in ((q, k), (q, k[:, :, :7]), (q, k.bfloat16()), (q[0], k)):
        with pytest.raises(ValueError):
            B.rope(*a, plan)
    with pytest.raises(ValueError):
        B.rope(q, k, plan, pos=torch.zeros(1, 8, dtype=torch.int64))


def check(got, x, p, plan, freq, **kw):
    want = ref.rope(x, p, freq, **kw)
    x = np64(x)
    n = len(freq)
    m = kw.get("mscale", 1.0)
    iu = np.arange(n) * 2 if kw.get("interleaved") else np.arange(n)
    iv = iu + (1 if kw.get("interleaved") else n)
    size = np.zeros_like(x)
    size[..., iu] = size[..., iv] = m * (np.abs(x[..., iu]) + np.abs(x[..., iv]))
    tol = 8 * 2.0 ** -24 * size + 1e-37
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(want)
    assert (np.abs(np64(got) - want) <= tol).all()


def positions(Bn, T, far, seed=0):
    g = np.random.default_rng(seed)
    p = g.integers(-far, far + 1, (Bn, T)).astype(np.int32)
    return p, torch.from_numpy(p).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", [  # B, H, Hkv, T, d, rot, far
    (1, 1, 1, 1, 2, 2, 5),
    (2, 4, 2, 33, 64, 64, 4096),
    (64, 20, 4, 1, 128, 128, 1 << 20),
    (1, 3, 1, 700, 96, 64, 131072),
    (3, 5, 5, 17, 256, 256, 1 << 30),
    (1, 2, 2, 9, 80, 24, 100),       # rot / 2 is no multiple of the vector
    (1, 2, 1, 9, 33, 30, 100),       # rows of odd length
    (1, 0, 2, 9, 64, 32, 100),       # keys alone
    (2, 16, 16, 1500, 128, 128, 8192),
])
def test_rope(shape, interleaved, inverse, dtype):
    Bn, H, Hkv, T, d, rot, far = shape
    g = torch.Generator().manual_seed(T + d)
    q, k = (torch.randn(Bn, h, T, d, generator=g).to(dtype).cuda() for h in (H, Hkv))
    how = dict(theta=10000.0, factor=4.0, original_length=2048.0)
    plan = B.rope_plan(rot, interleaved=interleaved, mscale=1.25, **how)
    freq = ref.rope_frequencies(rot, **how)
    p, pos = positions(Bn, T, far)
    qo, ko = B.rope(q, k, plan, pos=pos, inverse=inverse)
    for x, y in ((q, qo), (k, ko)):
        assert y.is_contiguous()
        check(y, x, p, plan, freq, interleaved=interleaved, inverse=inverse, mscale=1.25)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_strides_in_place_and_no_positions(dtype):
    """Slices of one [B, T, heads, d] projection, out of place, in place, and at odd offsets; positions 0..T-1."""
    Bn, H, Hkv, T, d = 2, 6, 3, 50, 64
    g = torch.Generator().manual_seed(1)
    plan, freq = B.rope_plan(d), ref.rope_frequencies(d)
    p = np.arange(T)[None].repeat(Bn, 0)
    for pad in (0, 1):       # an odd pitch: no 16-byte accesses
        buf = torch.randn(Bn, T, (H + 2 * Hkv) * d + pad, generator=g).to(dtype).cuda()
        keep = buf.clone()
        q = buf[..., :H * d].unflatten(-1, (H, d)).transpose(1, 2)
        k = buf[..., H * d:(H + Hkv) * d].unflatten(-1, (Hkv, d)).transpose(1, 2)
        want_q, want_k = q.clone(), k.clone()
        qo, ko = B.rope(q, k, plan)
        check(qo, want_q, p, plan, freq)
        check(ko, want_k, p, plan, freq)
        assert torch.equal(buf, keep)
        B.rope(q, k, plan, out=(q, k))
        assert torch.equal(q, qo) and torch.equal(k, ko)
        assert torch.equal(buf[..., (H + Hkv) * d:], keep[..., (H + Hkv) * d:])
    # one key head for all: an expanded input
    one = torch.randn(Bn, 1, T, d, generator=g).to(dtype).cuda()
    qo, ko = B.rope(one.expand(Bn, 4, T, d), one, plan)
    assert all(torch.equal(qo[:, h], ko[:, 0]) for h in range(4))


@pytest.mark.gpu
def test_there_and_back():
    q = torch.randn(1, 4, 300, 128, device="cuda")
    plan = B.rope_plan(128)
    _, pos = positions(1, 300, 1 << 30)
    a = B.rope(q, q[:, :1], plan, pos=pos)
    b, _ = B.rope(*a, plan, pos=pos, inverse=True)
    # two turns, each within 8 * 2^-24 of |u| + |v|
    assert (b - q).abs().max() <= 32 * 2.0 ** -24 * q.abs().max()
