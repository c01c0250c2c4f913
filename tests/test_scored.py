"""Scored attention (capped scores, distance bias, key ranges, shared key
heads): host checks on the CPU, parity with the float64 oracle on the GPU.

Tolerances: fp32 as every fp32 test (1e-5 of the largest value for O and LSE,
1e-4 for gradients). bf16: O per row as every bf16 test; LSE 1e-4 absolute
(products of bf16 values summed in fp32 over d <= 128 terms: 128 * 2^-24 of
sum |q k| ~ 10, then a few fp32 steps of values up to 50); gradients 5e-3 in
the Frobenius norm (P, dS, O in D and the result are each rounded to bf16,
uniformly within half a step of 2^-8: four times 2^-9 / sqrt(3) = 1.1e-3,
added in squares 2.3e-3).
"""
import math

import numpy as np
import pytest
import torch

import exact_tiled_softmax_attn_gb300 as B
from oracle import scored as ref

from parity import check_o, frob_rel, max_rel, np64


# ------------------------------------------------------------------ CPU

def test_oracle_gradients_are_differences():
    """The oracle's gradients against central differences of its own loss."""
    g = np.random.default_rng(0)
    q, k, v, do = (g.standard_normal(s) for s in ((1, 4, 5, 3), (1, 2, 7, 3), (1, 2, 7, 2), (1, 4, 5, 2)))
    how = dict(scale=0.7, softcap=1.5, slopes=g.standard_normal(4), q_pos=[[2, 3, 4, 5, 6]],
               key_begin=[[0, 1, 0, 9, 2]], key_end=[[3, 4, 7, 7, 7]], causal=True)
    r = ref.scored(q, k, v, do, **how)
    assert np.isneginf(r["LSE"][0, :, 3]).all() and not r["dQ"][0, :, 3].any()
    for x, name in ((q, "dQ"), (k, "dK"), (v, "dV")):
        for at in np.ndindex(*x.shape):
            h = 1e-6
            old = x[at]
            loss = []
            for s in (1, -1):
                x[at] = old + s * h
                loss.append((ref.scored(q, k, v, **how)["O"] * do).sum())
            x[at] = old
            assert abs((loss[0] - loss[1]) / (2 * h) - r[name][at]) < 1e-7


def _fwd(score=None, **kw):
    a = dict(Q=0x100000, K=0x200000, V=0x300000, O=0x400000, LSE=0x500000, B=1, H=4, Hkv=2, Tq=8, Tk=8, d=64, dv=64,
             scale=0.125, score=score, dtype=B.ATTN_BF16, workspace=0x9000000, workspace_bytes=1 << 20, stream=0,
             check=False)
    a.update(kw)
    return B.attn_fwd_scored(**a)


BAD = [
    (dict(B=-1), B.ATTN_ERR_INVALID_ARG),
    (dict(Hkv=0), B.ATTN_ERR_INVALID_ARG),
    (dict(Hkv=3), B.ATTN_ERR_INVALID_ARG),
    (dict(scale=0.0), B.ATTN_ERR_INVALID_ARG),
    (dict(scale=float("nan")), B.ATTN_ERR_INVALID_ARG),
    (dict(dtype=5), B.ATTN_ERR_INVALID_ARG),
    (dict(d=136), B.ATTN_ERR_UNSUPPORTED),
    (dict(dv=60), B.ATTN_ERR_UNSUPPORTED),
    (dict(dtype=B.ATTN_F32, dv=129), B.ATTN_ERR_UNSUPPORTED),
    (dict(Tk=(1 << 30) + 1), B.ATTN_ERR_INVALID_ARG),
    (dict(Tq=1 << 30), B.ATTN_ERR_INVALID_ARG),               # 2 heads a group: more than 2^30 packed rows
    (dict(B=1 << 20, Hkv=1 << 11, H=1 << 11), B.ATTN_ERR_INVALID_ARG),
    (dict(Q=None), B.ATTN_ERR_INVALID_ARG),
    (dict(K=0x200008), B.ATTN_ERR_MISALIGNED),
    (dict(workspace=None), B.ATTN_ERR_WORKSPACE),
    (dict(workspace_bytes=64), B.ATTN_ERR_WORKSPACE),
    (dict(workspace=0x9000010), B.ATTN_ERR_WORKSPACE),
    (dict(score=B.AttnScore(-1.0, 0, 0, 0, 0, 0)), B.ATTN_ERR_INVALID_ARG),
    (dict(score=B.AttnScore(float("inf"), 0, 0, 0, 0, 0)), B.ATTN_ERR_INVALID_ARG),
    (dict(score=B.AttnScore(1e-5, 0, 0, 0, 0, 0)), B.ATTN_ERR_INVALID_ARG),
    (dict(score=B.AttnScore(2e6, 0, 0, 0, 0, 0)), B.ATTN_ERR_INVALID_ARG),
    (dict(score=B.AttnScore(float("nan"), 0, 0, 0, 0, 0)), B.ATTN_ERR_INVALID_ARG),
    (dict(score=B.AttnScore(0.0, 2, 0, 0, 0, 0)), B.ATTN_ERR_INVALID_ARG),
    (dict(score=B.AttnScore(0.0, 0, 0x600002, 0, 0, 0)), B.ATTN_ERR_MISALIGNED),
    (dict(score=B.AttnScore(0.0, 0, 0, 0, 0, 0x600001)), B.ATTN_ERR_MISALIGNED),
]


@pytest.mark.parametrize("kw,status", BAD + [
    (dict(O=0x200000), B.ATTN_ERR_INVALID_ARG),                 # output over K
    (dict(LSE=0x400000), B.ATTN_ERR_INVALID_ARG),
    (dict(workspace=0x100000), B.ATTN_ERR_WORKSPACE),
    (dict(score=B.AttnScore(0.0, 0, 0, 0x400000, 0, 0)), B.ATTN_ERR_INVALID_ARG),   # output over q_pos
    (dict(score=B.AttnScore(0.0, 0, 0x9000000, 0, 0, 0)), B.ATTN_ERR_WORKSPACE),    # workspace over slopes
])
def test_forward_refusals(kw, status):
    assert _fwd(**kw) == status


def _bwd(score=None, **kw):
    a = dict(Q=0x100000, K=0x200000, V=0x300000, O=0x400000, LSE=0x500000, dO=0x600000, dQ=0x700000, dK=0x800000,
             dV=0x900000, B=1, H=4, Hkv=2, Tq=8, Tk=8, d=64, dv=64, scale=0.125, score=score, dtype=B.ATTN_BF16,
             workspace=0x9000000, workspace_bytes=1 << 20, stream=0, check=False)
    a.update(kw)
    return B.attn_bwd_scored(**a)


@pytest.mark.parametrize("kw,status", BAD + [
    (dict(dQ=0x600000), B.ATTN_ERR_INVALID_ARG),
    (dict(dK=0x900000), B.ATTN_ERR_INVALID_ARG),
    (dict(dO=None), B.ATTN_ERR_INVALID_ARG),
    (dict(workspace=0x800000), B.ATTN_ERR_WORKSPACE),
    (dict(score=B.AttnScore(0.0, 0, 0, 0, 0x700000, 0)), B.ATTN_ERR_INVALID_ARG),
])
def test_backward_refusals(kw, status):
    # (an output over another output is refused with the workspace's own check first where it is the workspace)
    assert _bwd(**kw) in ((status, B.ATTN_ERR_WORKSPACE) if "workspace" in kw else (status,))


def test_nothing_to_do_needs_no_device():
    assert _fwd(B=0) == B.ATTN_OK
    assert _fwd(Tq=0, workspace=None) == B.ATTN_OK
    assert _fwd(H=0) == B.ATTN_OK
    assert _bwd(B=0, workspace=None) == B.ATTN_OK
    for f in (B.attn_fwd_scored_workspace_size, B.attn_bwd_scored_workspace_size):
        assert f(1, 4, 2, 0, 8, 64, 64, B.ATTN_BF16) == 0
        assert f(1, 4, 2, 8, 0, 64, 64, B.ATTN_BF16) == 0
        assert f(1, 4, 3, 8, 8, 64, 64, B.ATTN_BF16) == 0
        assert f(1, 4, 2, 8, 8, 64, 64, B.ATTN_BF16) > 0


def test_wrapper_refusals():
    q, k = torch.zeros(1, 4, 8, 64), torch.zeros(1, 2, 8, 64)
    with pytest.raises(ValueError):
        B.forward_scored(q, k, k)   # not on a GPU
    for bad in (dict(q_pos=torch.zeros(1, 8)), dict(key_end=torch.zeros(1, 7, dtype=torch.int32)),
                dict(slopes=torch.zeros(3)), dict(slopes=torch.zeros(4, dtype=torch.float64)),
                dict(key_begin=torch.zeros(8, 2, dtype=torch.int32).t()[:1])):
        with pytest.raises(ValueError):
            B.forward_scored(q, k, k, **bad)
    with pytest.raises(ValueError):
        B.forward_scored(q, torch.zeros(1, 3, 8, 64), torch.zeros(1, 3, 8, 64))
    with pytest.raises(ValueError):
        B.forward_scored(q.transpose(2, 3), k, k)
    with pytest.raises(ValueError):
        B.forward_scored(q, k, k.bfloat16())


# ------------------------------------------------------------------ GPU

def arrays(mask, Bn, Tq, Tk, seed=0):
    """key_begin, key_end, q_pos as numpy int32 [B, Tq], or None."""
    g = np.random.default_rng(seed)
    i = np.arange(Tq)[None] + np.zeros((Bn, 1), np.int64)
    pos = i + Tk - Tq
    begin = end = None
    if mask == "docs":
        cut = np.sort(g.integers(0, Tk + 1, (Bn, 4)), axis=1)
        doc = (np.clip(pos, 0, Tk - 1)[:, :, None] >= cut[:, None, :]).sum(-1)
        edge = np.concatenate([np.zeros((Bn, 1), np.int64), cut, np.full((Bn, 1), Tk)], axis=1)
        begin = np.take_along_axis(edge, doc, 1)
        end = np.minimum(np.take_along_axis(edge, doc + 1, 1), pos + 1)
    elif mask == "prefix":
        end = np.maximum(pos + 1, Tk // 3)
    elif mask == "window":
        begin, end = pos - 70, pos + 1
    elif mask == "causal":
        end = pos + 1
    elif mask == "wild":        # any ranges in any order, empty ones and ones outside [0, Tk) among them
        begin, end = g.integers(-9, Tk + 9, (Bn, Tq)), g.integers(-9, Tk + 40, (Bn, Tq))
        pos = g.integers(-300, Tk + 300, (Bn, Tq))
    elif mask == "empty":
        begin, end = np.full((Bn, Tq), 3), np.full((Bn, Tq), 3)
    elif mask == "some":        # whole tiles of padding rows, then one row
        begin, end = np.zeros((Bn, Tq), np.int64), np.where(i % 300 > 140, 0, Tk)
    as32 = lambda x: None if x is None else x.astype(np.int32)  # noqa: E731
    return as32(begin), as32(end), as32(pos)


def make(Bn, H, Hkv, Tq, Tk, d, dv, dtype, seed, grad=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = [2.0 * r(Bn, H, Tq, d), r(Bn, Hkv, Tk, d), r(Bn, Hkv, Tk, dv)] + ([r(Bn, H, Tq, dv)] if grad else [])
    return [t.to(dtype).cuda() for t in x]


def check_lse(lse, want, dtype):
    lse = np64(lse)
    inf = np.isneginf(want)
    assert np.array_equal(np.isneginf(lse), inf)
    if (~inf).any():
        err = np.abs(lse[~inf] - want[~inf]).max()
        assert err <= (1e-5 * max(1.0, np.abs(want[~inf]).max()) if dtype == torch.float32 else 1e-4), err


def check_grad(g, want, dtype, name):
    assert np.isfinite(np64(g)).all(), name
    err = max_rel(g, want) if dtype == torch.float32 else frob_rel(g, want)
    assert err <= (1e-4 if dtype == torch.float32 else 5e-3), (name, err)


def how_of(mask, cap, bias, Bn, H, Tq, Tk, seed=1):
    begin, end, pos = arrays(mask, Bn, Tq, Tk, seed)
    gpu = lambda x: None if x is None else torch.from_numpy(x).cuda()  # noqa: E731
    slopes = torch.exp2(-8.0 * torch.arange(1, H + 1) / H).cuda() if bias else None
    return dict(softcap=cap, slopes=slopes, q_pos=gpu(pos), key_begin=gpu(begin), key_end=gpu(end))


def run_case(shape, mask, cap, bias, dtype, grad, causal=False, scale=None):
    Bn, H, Hkv, Tq, Tk, d, dv = shape
    x = make(*shape, dtype, seed=Tq + 3 * Tk + d, grad=grad)
    how = how_of(mask, cap, bias, Bn, H, Tq, Tk)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o, lse = B.forward_scored(*x[:3], causal=causal, scale=scale, **how)
    g = B.backward_scored(*x[:3], o, lse, x[3], causal=causal, scale=scale, **how) if grad else ()
    torch.cuda.synchronize()
    assert B.attn_device_status() == B.ATTN_OK
    r = ref.scored(*x, scale=scale, causal=causal, **how)
    check_o(o, r["O"], dtype)
    check_lse(lse, r["LSE"], dtype)
    for t, name in zip(g, ("dQ", "dK", "dV")):
        check_grad(t, r[name], dtype, name)


TYPES = [torch.float32, torch.bfloat16]
SHAPES = [  # B, H, Hkv, Tq, Tk, d, dv
    (1, 1, 1, 1, 1, 64, 64),
    (2, 4, 2, 130, 130, 64, 64),
    (1, 6, 2, 200, 333, 128, 128),
    (2, 3, 1, 129, 257, 40, 128),
    (1, 4, 4, 300, 300, 96, 64),
    (1, 8, 1, 37, 500, 128, 128),
    (1, 2, 1, 513, 100, 80, 80),
    (1, 2, 2, 640, 640, 128, 128),
    (1, 8, 1, 300, 260, 64, 64),      # long lists of row tiles for few key tiles: cut into parts
    (2, 6, 1, 500, 200, 128, 80),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("mask,cap,bias", [("none", 0.0, False), ("causal", 5.0, False), ("docs", 0.0, True),
                                           ("prefix", 3.0, True), ("window", 0.0, False), ("wild", 2.0, True),
                                           ("some", 0.0, False)])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_and_backward(shape, mask, cap, bias, dtype):
    run_case(shape, mask, cap, bias, dtype, grad=True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 4, 2, 70, 90, 64, 64), (1, 2, 2, 300, 129, 128, 128)])
def test_causal_flag_is_top_left(shape, dtype):
    """causal = 1 without positions blocks j > i, as attn_fwd does; rows past Tk see every key."""
    Bn, H, Hkv, Tq, Tk, d, dv = shape
    x = make(*shape, dtype, 3)
    o, lse = B.forward_scored(*x[:3], causal=True)
    r = ref.scored(*x, scale=1.0 / math.sqrt(d), causal=True)
    check_o(o, r["O"], dtype)
    check_lse(lse, r["LSE"], dtype)
    for t, name in zip(B.backward_scored(*x[:3], o, lse, x[3], causal=True), ("dQ", "dK", "dV")):
        check_grad(t, r[name], dtype, name)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "bf16"])
def test_rows_that_see_nothing(dtype):
    x = make(1, 2, 1, 150, 200, 64, 64, dtype, 5)
    how = how_of("empty", 4.0, True, 1, 2, 150, 200)
    o, lse = B.forward_scored(*x[:3], **how)
    g = B.backward_scored(*x[:3], o, lse, x[3], **how)
    assert not o.any() and torch.isneginf(lse).all()
    assert not any(t.any() for t in g)
    # no keys at all, and no queries
    o, lse = B.forward_scored(x[0], x[1][:, :, :0], x[2][:, :, :0])
    assert not o.any() and torch.isneginf(lse).all()
    e = x[0][:, :, :0]
    dq, dk, dv = B.backward_scored(e, x[1], x[2], e, lse[:, :, :0], e)
    assert dq.numel() == 0 and not dk.any() and not dv.any()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("mask,cap,bias", [("causal", 4.0, False), ("window", 0.0, True), ("wild", 0.0, False),
                                           ("some", 3.0, True)])
@pytest.mark.parametrize("shape", [(1, 2, 1, 150, 3000, 128, 128), (1, 1, 1, 300, 2100, 64, 64),
                                   (2, 3, 1, 100, 1500, 96, 128)])
def test_few_rows_against_many_keys(shape, mask, cap, bias, dtype):
    """More rows than the few-row kernel takes, too few to fill the GPU: the keys are cut into ranges."""
    run_case(shape, mask, cap, bias, dtype, grad=True)


@pytest.mark.gpu
def test_long_runs_of_idle_row_tiles():
    """Most row tiles of every head see nothing, in runs longer than any queue between a kernel's warps; the live rows
    give what they give without the idle ones (bit for bit, except for the order in dK's and dV's sums)."""
    H, Tq, Tk, d = 64, 5000, 2200, 64
    q, k, v, do = make(1, H, H, Tq, Tk, d, d, torch.bfloat16, 23)
    live = (torch.arange(Tq) // 256) % 7 == 0
    end = torch.where(live, Tk, 0).to(torch.int32)[None].cuda()
    idx = live.nonzero()[:, 0].cuda()
    o, lse = B.forward_scored(q, k, v, key_end=end)
    dq, dk, dv = B.backward_scored(q, k, v, o, lse, do, key_end=end)
    assert B.attn_device_status() == B.ATTN_OK
    qc, doc = q[:, :, idx].contiguous(), do[:, :, idx].contiguous()
    oc, lsec = B.forward_scored(qc, k, v)
    gc = B.backward_scored(qc, k, v, oc, lsec, doc)
    assert B.attn_device_status() == B.ATTN_OK
    assert torch.equal(o[:, :, idx], oc) and torch.equal(lse[:, :, idx], lsec) and torch.equal(dq[:, :, idx], gc[0])
    rest = (~live).nonzero()[:, 0].cuda()
    assert not o[:, :, rest].any() and not dq[:, :, rest].any() and torch.isneginf(lse[:, :, rest]).all()
    for a, b in ((dk, gc[1]), (dv, gc[2])):
        assert frob_rel(a, b) <= 5e-3


@pytest.mark.gpu
@pytest.mark.parametrize("mask", ["causal", "wild"])
def test_shared_key_heads_equal_repeated_ones(mask):
    """16 query heads on 2 key heads, whose row tiles are cut into parts, against 16 key heads with repeated keys."""
    H, Hkv, T, d = 16, 2, 2048, 64
    q, k, v, do = make(1, H, Hkv, T, T, d, d, torch.bfloat16, 29)
    how = how_of(mask, 0.0, True, 1, H, T, T)
    o, lse = B.forward_scored(q, k, v, **how)
    dq, dk, dv = B.backward_scored(q, k, v, o, lse, do, **how)
    assert B.attn_device_status() == B.ATTN_OK
    kr, vr = (t.repeat_interleave(H // Hkv, 1) for t in (k, v))
    o2, lse2 = B.forward_scored(q, kr, vr, **how)
    dq2, dk2, dv2 = B.backward_scored(q, kr, vr, o2, lse2, do, **how)
    assert B.attn_device_status() == B.ATTN_OK
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and torch.equal(dq, dq2)
    for a, b in ((dk, dk2), (dv, dv2)):
        # each of the repeated heads' gradients is rounded once more
        assert frob_rel(a, b.double().view(1, Hkv, H // Hkv, T, d).sum(2)) <= 5e-3


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("Tq,Tk", [(1, 5000), (3, 700), (200, 700)])
def test_unused_cache_rows_may_hold_anything(Tq, Tk, dtype):
    """NaN and infinities before and behind a batch entry's ranges change nothing."""
    lens = [Tk // 3 + 1, Tk - 5]
    x = make(2, 8, 2, Tq, Tk, 64, 128, dtype, 7, grad=False)
    begin = torch.full((2, Tq), 11, dtype=torch.int32, device="cuda")
    end = torch.tensor(lens, dtype=torch.int32, device="cuda")[:, None].expand(2, Tq).contiguous()
    o, lse = B.forward_scored(*x, key_begin=begin, key_end=end)
    for b in range(2):
        for t, junk in ((x[1], float("inf")), (x[2], float("nan"))):
            t[b, :, :11] = junk
            t[b, :, lens[b]:] = junk
    o2, lse2 = B.forward_scored(*x, key_begin=begin, key_end=end)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("shape,mask,cap,bias", [
    ((1, 8, 8, 1, 3000, 128, 128), "causal", 5.0, False),
    ((3, 8, 2, 1, 1111, 64, 64), "window", 0.0, True),
    ((2, 16, 2, 3, 2500, 128, 64), "causal", 0.0, False),
    ((1, 14, 2, 5, 777, 96, 96), "wild", 3.0, True),
    ((40, 4, 1, 2, 300, 40, 40), "causal", 0.0, True),
    ((1, 64, 1, 5, 2000, 128, 128), "causal", 0.0, False),
    ((2, 2, 2, 1, 15, 64, 128), "none", 0.0, False),
])
def test_tokens_against_a_cache(shape, mask, cap, bias, dtype):
    run_case(shape, mask, cap, bias, dtype, grad=False)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("cap", [0.5, 5.0, 50.0])
def test_scores_far_beyond_the_cap(cap, dtype):
    """Scores up to several hundred: the cap flattens them, and its derivative vanishes."""
    run_case((1, 2, 1, 140, 300, 64, 64), "causal", cap, False, dtype, grad=True, scale=4.0)


@pytest.mark.gpu
def test_bias_at_far_positions():
    """The bias depends on the distance alone: equal at positions near 0 and near 2^20."""
    x = make(1, 4, 2, 5, 400, 64, 64, torch.bfloat16, 9, grad=False)
    r = None
    for Tk, at in ((400, 0),):
        how = how_of("causal", 0.0, True, 1, 4, 5, Tk)
        r = B.forward_scored(*x, **how)
    k, v = (torch.zeros(1, 2, (1 << 20) + 400, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k[:, :, 1 << 20:], v[:, :, 1 << 20:] = x[1], x[2]
    far = dict(how, q_pos=how["q_pos"] + (1 << 20), key_end=how["key_end"] + (1 << 20),
               key_begin=torch.full((1, 5), 1 << 20, dtype=torch.int32, device="cuda"))
    o, lse = B.forward_scored(x[0], k, v, **far)
    assert (lse - r[1]).abs().max() <= 1e-4
    assert (o.float() - r[0].float()).abs().max() <= 2.0 ** -7 * r[0].float().abs().max()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "bf16"])
def test_repeats_are_bitwise_equal_and_replay_from_a_graph(dtype):
    """Two eager calls and replays of a captured forward and backward give equal bits; the graph follows new inputs."""
    shape = (2, 6, 2, 260, 260, 64, 64)
    x = make(*shape, dtype, 11)
    how = how_of("docs", 5.0, True, 2, 6, 260, 260)

    def both():
        o, lse = B.forward_scored(*x[:3], **how)
        return [o, lse, *B.backward_scored(*x[:3], o, lse, x[3], **how)]

    a, b = both(), both()
    torch.cuda.synchronize()
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        c = both()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(s, t) for s, t in zip(a, c))
    x[0].copy_(make(*shape, dtype, 12)[0])
    d = both()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(s, t) for s, t in zip(d, c)) and not torch.equal(a[0], d[0])


@pytest.mark.gpu
def test_on_another_stream():
    x = make(1, 4, 2, 300, 300, 64, 64, torch.bfloat16, 13)
    want = B.forward_scored(*x[:3], causal=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        o, lse = B.forward_scored(*x[:3], causal=True, stream=stream)
        g = B.backward_scored(*x[:3], o, lse, x[3], causal=True, stream=stream)
        s.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1]) and all(t.isfinite().all() for t in g)


@pytest.mark.gpu
def test_guard_rows_stay_as_they_were():
    """Nothing is written behind the outputs or the stated workspace."""
    Bn, H, Hkv, Tq, Tk, d, dv = 1, 4, 2, 131, 140, 72, 40
    for dt, code in ((torch.bfloat16, B.ATTN_BF16), (torch.float32, B.ATTN_F32)):
        x = make(Bn, H, Hkv, Tq, Tk, d, dv, dt, 17)

        def guarded(n, dtype):
            return torch.full((n + 4096,), 7.0, dtype=dtype, device="cuda")
        o, lse = guarded(Bn * H * Tq * dv, dt), guarded(Bn * H * Tq, torch.float32)
        dq, dk, dv_ = (guarded(t.numel(), dt) for t in x[:3])
        nf, nb = (f(Bn, H, Hkv, Tq, Tk, d, dv, code) for f in (B.attn_fwd_scored_workspace_size,
                                                              B.attn_bwd_scored_workspace_size))
        ws = torch.full((max(nf, nb) + 4096,), 7, dtype=torch.uint8, device="cuda")
        sc = B.AttnScore(0.0, 1, 0, 0, 0, 0)
        B.attn_fwd_scored(*x[:3], o, lse, Bn, H, Hkv, Tq, Tk, d, dv, 0.1, sc, code, ws, nf)
        torch.cuda.synchronize()
        assert (ws[nf:] == 7).all()
        B.attn_bwd_scored(*x[:3], o, lse, x[3], dq, dk, dv_, Bn, H, Hkv, Tq, Tk, d, dv, 0.1, sc, code, ws, nb)
        torch.cuda.synchronize()
        assert (ws[nb:] == 7).all()
        for t, n in ((o, Bn * H * Tq * dv), (lse, Bn * H * Tq), (dq, x[0].numel()), (dk, x[1].numel()),
                     (dv_, x[2].numel())):
            assert (t[n:] == 7.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "bf16"])
def test_rope_then_attention_then_both_gradients(dtype):
    """A layer's use: rotary positions, capped attention over documents, and the gradients back to the unrotated
    queries and keys, against the same chain in float64."""
    Bn, H, Hkv, T, d = 2, 6, 2, 270, 64
    q, k, v, do = make(Bn, H, Hkv, T, T, d, d, dtype, 19)
    how = how_of("docs", 6.0, False, Bn, H, T, T)
    plan = B.rope_plan(48, theta=500.0)
    pos = how["q_pos"]
    qr, kr = B.rope(q, k, plan, pos=pos)
    o, lse = B.forward_scored(qr, kr, v, **how)
    dqr, dkr, dv = B.backward_scored(qr, kr, v, o, lse, do, **how)
    dq, dk = B.rope(dqr, dkr, plan, pos=pos, inverse=True)
    f = ref.rope_frequencies(48, theta=500.0)
    p = pos.cpu().numpy()
    # the chain in float64 from what the attention was given: the rotated values as they were rounded
    r = ref.scored(qr, kr, v, do, scale=1.0 / math.sqrt(d), **how)
    check_o(o, r["O"], dtype)
    check_grad(dq, ref.rope(r["dQ"], p, f, inverse=True), dtype, "dQ")
    check_grad(dk, ref.rope(r["dK"], p, f, inverse=True), dtype, "dK")
    check_grad(dv, r["dV"], dtype, "dV")
    # a half step of the type for each of the two products' sums
    bound = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -21
    assert np.abs(np64(qr) - ref.rope(q, p, f)).max() <= bound * np64(q).__abs__().max() * 1.5


# ------------------------------------------------------------------ what no query reads, and what one does

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (4.0, False), (0.0, True), (4.0, True)])
@pytest.mark.parametrize("shape", [(2, 4, 2, 300, 420, 64, 64), (2, 4, 1, 300, 420, 128, 128), (1, 2, 2, 20, 300, 72, 40),
                                   (1, 16, 1, 130, 260, 64, 64)])
def test_padding_may_hold_anything(shape, cap, bias, dtype):
    """A padded batch: queries that see no key and keys that no query sees are NaN and infinite, and every result is
    what it is with finite padding (bit for bit, except for the roundings of a cap)."""
    Bn, H, Hkv, Tq, Tk, d, dv = shape
    x = make(*shape, dtype, 31)
    how = how_of("none", cap, bias, Bn, H, Tq, Tk)
    live = torch.tensor([Tq - 9, Tq // 2 + 3][:Bn])[:, None]
    i = torch.arange(Tq)[None]
    begin = torch.full((Bn, Tq), 13).where(i < 40, torch.tensor(21))
    end = torch.where(i < live, Tk - 30 + torch.arange(Bn)[:, None], 0)
    how["key_begin"], how["key_end"] = (t.to(torch.int32).cuda() for t in (begin, end))

    def both():
        o, lse = B.forward_scored(*x[:3], **how)
        oj = o.clone()
        for b in range(Bn):
            oj[b, :, live[b, 0]:] = junk
        g = B.backward_scored(*x[:3], oj, lse, x[3], **how)
        assert B.attn_device_status() == B.ATTN_OK
        return [o, lse, *g]
    junk = 0.0
    want = both()
    assert all(t.isfinite().all() for t in want[2:])
    for junk in (float("nan"), float("inf")):
        for b in range(Bn):
            x[0][b, :, live[b, 0]:] = junk
            x[3][b, :, live[b, 0]:] = junk
            for t in x[1:3]:
                t[b, :, :13] = junk
                t[b, :, Tk - 30 + b:] = junk
        got = both()
        for a, c, name in zip(got, want, ("O", "LSE", "dQ", "dK", "dV")):
            if dtype == torch.bfloat16 and cap:   # the largest score near by decides how the cap is evaluated
                check_lse(a, np64(c), dtype) if name == "LSE" else check_grad(a, np64(c), dtype, name)
            else:
                assert torch.equal(a, c), (name, junk)
    for b in range(Bn):
        assert not got[2][b, :, live[b, 0]:].any()
        assert not got[3][b, :, :13].any() and not got[4][b, :, Tk - 30 + b:].any()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("cap", [0.0, 5.0])
@pytest.mark.parametrize("shape", [(1, 2, 2, 1, 700, 64, 64), (2, 8, 2, 3, 50, 128, 128), (1, 2, 1, 300, 3000, 64, 64),
                                   (2, 40, 40, 300, 300, 128, 128)])
def test_a_nan_that_a_row_sees_shows(shape, cap, dtype):
    Bn, H, Hkv, Tq, Tk, d, dv = shape
    x = make(*shape, dtype, 37, grad=False)
    want = B.forward_scored(*x, softcap=cap)
    x[0][-1, 1, Tq // 2, 3] = float("nan")
    o, lse = B.forward_scored(*x, softcap=cap)
    assert o[-1, 1, Tq // 2].isnan().all() and lse[-1, 1, Tq // 2].isnan()
    o[-1, 1, Tq // 2], lse[-1, 1, Tq // 2] = want[0][-1, 1, Tq // 2], want[1][-1, 1, Tq // 2]
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


# ------------------------------------------------------------------ slopes, positions, row counts

def magnitudes(x, how, scale):
    """Sums of absolute values behind each result: what a relative error of every term is an error of."""
    q, k, v, do = (np64(t) for t in x)
    G = q.shape[1] // k.shape[1]
    k, v = np.repeat(k, G, 1), np.repeat(v, G, 1)
    r = ref.scored(*x, scale=scale, **how)
    j = np.arange(k.shape[2])
    get = lambda t, default: default if t is None else np64(t)[:, None, :, None]  # noqa: E731
    pos = get(how["q_pos"], np.arange(q.shape[2])[None, None, :, None])
    s = scale * q @ k.swapaxes(2, 3)
    if how["softcap"]:
        s = how["softcap"] * np.tanh(s / how["softcap"])
    s = s - np64(how["slopes"])[None, :, None, None] * np.abs(pos - j)
    seen = (j >= get(how["key_begin"], 0)) & (j < get(how["key_end"], len(j)))
    p = np.where(seen, np.exp(np.minimum(s - np.where(np.isneginf(r["LSE"]), 0, r["LSE"])[..., None], 0)), 0)
    a = np.abs
    ds = p * (a(do) @ a(v).swapaxes(2, 3) + (a(do) * a(r["O"])).sum(-1, keepdims=True))
    group = lambda t: t.reshape(t.shape[0], -1, G, *t.shape[2:]).sum(2)  # noqa: E731
    return {"score": scale * (a(q) @ a(k).swapaxes(2, 3)).max(), "O": p @ a(v), "dQ": scale * ds @ a(k),
            "dK": group(scale * ds.swapaxes(2, 3) @ a(q)), "dV": group(p.swapaxes(2, 3) @ a(do))}


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("mask,cap,scale", [("causal", 0.0, None), ("wild", 0.0, None), ("wild", 0.7, 4.0), ("none", 2.0, 0.05)])
@pytest.mark.parametrize("shape", [(1, 6, 2, 200, 300, 64, 64), (2, 6, 3, 9, 400, 128, 64), (1, 6, 1, 150, 2000, 64, 64)])
def test_slopes_of_any_size_and_sign(shape, mask, cap, scale, dtype):
    """Steep slopes leave a row a key or two; negative ones prefer far keys; 0 is none."""
    Bn, H, Hkv, Tq, Tk, d, dv = shape
    x = make(*shape, dtype, 41)
    how = how_of(mask, cap, False, Bn, H, Tq, Tk)
    how["slopes"] = torch.tensor([4.0, -0.5, 0.0, 9.0, 0.25, -0.01], device="cuda")
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o, lse = B.forward_scored(*x[:3], scale=scale, **how)
    g = B.backward_scored(*x[:3], o, lse, x[3], scale=scale, **how)
    assert B.attn_device_status() == B.ATTN_OK
    r, size = ref.scored(*x, scale=scale, **how), magnitudes(x, how, scale)
    # A score is off by the sum of its products (d roundings of sums up to `size`) and by a few half steps of its bias
    # (up to |slope| times the distance, in log2 units; with ranges of any kind a row's keys may all lie far off).
    far = (9.0 if mask == "wild" else 0.5) * (Tk + 600) * 1.4427
    score = d * 2.0 ** -24 * size["score"] + 6 * far * 2.0 ** -24
    half = 0.0 if dtype == torch.float32 else 2.0 ** -8
    terms = max(Tk, H // Hkv * Tq, d) * 2.0 ** -24   # roundings of a sum
    inf = np.isneginf(r["LSE"])
    assert np.array_equal(np.isneginf(np64(lse)), inf)
    assert np.abs(np64(lse)[~inf] - r["LSE"][~inf]).max() <= 1e-4 + score
    # weights off by the score's and the sum's error, rounded once; the result rounded once
    assert (np.abs(np64(o) - r["O"]) <= (2 * score + terms + 1e-5 + half) * size["O"] + half * np.abs(r["O"]) + 1e-6).all()
    # P T, dS, the O in D and the result are rounded; T is off by the score's error over the cap
    rel = 3 * half + 4 * score + terms + 1e-5 + (2 * score / cap if cap else 0.0)
    for t, name in zip(g, ("dQ", "dK", "dV")):
        assert (np.abs(np64(t) - r[name]) <= rel * size[name] + half * np.abs(r[name]) + 1e-6).all(), name


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(2, 12, 1, 5, 900, 64, 128), (1, 4, 1, 16, 500, 128, 40), (1, 2, 2, 64, 130, 64, 64),
                                   (1, 5, 1, 13, 700, 64, 64), (1, 11, 1, 3, 64, 128, 128), (1, 1, 1, 17, 1, 64, 64)])
@pytest.mark.parametrize("mask,cap,bias", [("wild", 3.0, True), ("causal", 0.0, False)])
def test_row_counts_of_the_few_row_kernel(shape, mask, cap, bias):
    run_case(shape, mask, cap, bias, torch.bfloat16, grad=False)


@pytest.mark.gpu
@pytest.mark.parametrize("Bn,H,Hkv,Tq", [(700, 4, 2, 1), (700, 8, 1, 3), (1200, 1, 1, 40)])
def test_more_sequences_than_threads(Bn, H, Hkv, Tq):
    """Sequences of very different lengths, many without a key: every one against a call of its own kind in float64."""
    Tk, d = 190, 64
    x = make(Bn, H, Hkv, Tq, Tk, d, d, torch.bfloat16, 43, grad=False)
    g = torch.Generator().manual_seed(44)
    n = torch.randint(1, Tk + 1, (Bn, 1), generator=g)
    n[torch.rand(Bn, 1, generator=g) < 0.4] = 0
    n[-40:] = 0
    n[:3] = 0
    end = n.expand(Bn, Tq).to(torch.int32).contiguous().cuda()
    o, lse = B.forward_scored(*x, key_end=end)
    assert B.attn_device_status() == B.ATTN_OK
    r = ref.scored(*x, scale=1.0 / math.sqrt(d), key_end=end)
    check_o(o, r["O"], torch.bfloat16)
    check_lse(lse, r["LSE"], torch.bfloat16)


# ------------------------------------------------------------------ graphs, streams, long caches

@pytest.mark.gpu
def test_a_decoding_step_replays_from_a_graph():
    """One captured call serves a growing sequence: the lengths are device memory."""
    q, k, v = make(3, 8, 2, 1, 2000, 128, 128, torch.bfloat16, 47, grad=False)
    end = torch.tensor([[5], [700], [64]], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    B.forward_scored(q, k, v, key_end=end)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        o, lse = B.forward_scored(q, k, v, key_end=end)
    for lens in ((5, 700, 64), (2000, 0, 65), (1, 1999, 1000)):
        end.copy_(torch.tensor(lens, dtype=torch.int32)[:, None])
        graph.replay()
        want = B.forward_scored(q, k, v, key_end=end)
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert B.attn_device_status() == B.ATTN_OK


@pytest.mark.gpu
def test_two_streams_at_once():
    """Calls on two streams, each with its own workspace, overlap without a trace in the results."""
    sets = [make(2, 8, 2, 520, 520, 64, 64, torch.bfloat16, s) for s in (51, 52)]
    tok = [make(4, 8, 2, 1, 3000, 64, 64, torch.bfloat16, s, grad=False) for s in (53, 54)]

    def work(i):
        o, lse = B.forward_scored(*sets[i][:3], causal=True, softcap=5.0)
        return [o, lse, *B.backward_scored(*sets[i][:3], o, lse, sets[i][3], causal=True, softcap=5.0),
                *B.forward_scored(*tok[i])]
    want = [work(0), work(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(6):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i].append(work(i))
    torch.cuda.synchronize()
    assert B.attn_device_status() == B.ATTN_OK
    for i in (0, 1):
        for run in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(run, want[i]))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,Tq", [(torch.bfloat16, 1), (torch.bfloat16, 150), (torch.float32, 3)])
def test_offsets_beyond_32_bits(dtype, Tq):
    """The last key head of the last sequence lies behind element 2^31 of the cache, its last keys far behind its first."""
    Bn, H, Hkv, Tk, d = 2, 8, 4, (1 << 22) + 5, 128
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    q = make(Bn, H, Hkv, Tq, 1, d, d, dtype, 57, grad=False)[0]
    k, v = (torch.empty(Bn, Hkv, Tk, d, dtype=dtype, device="cuda") for _ in range(2))
    n = 777
    g = torch.Generator().manual_seed(58)
    kn, vn = (torch.randn(Bn, Hkv, n, d, generator=g).to(dtype).cuda() for _ in range(2))
    k[:, :, Tk - n:], v[:, :, Tk - n:] = kn, vn
    begin = torch.full((Bn, Tq), Tk - n, dtype=torch.int32, device="cuda")
    o, lse = B.forward_scored(q, k, v, key_begin=begin)
    assert B.attn_device_status() == B.ATTN_OK
    r = ref.scored(q, kn, vn, scale=1.0 / math.sqrt(d))
    check_o(o, r["O"], dtype)
    check_lse(lse, r["LSE"], dtype)
    if Tq == 150:
        do = make(Bn, H, Hkv, Tq, 1, d, d, dtype, 59)[3]
        dq, dk, dv = B.backward_scored(q, k, v, o, lse, do, key_begin=begin)
        assert B.attn_device_status() == B.ATTN_OK
        r = ref.scored(q, kn, vn, do, scale=1.0 / math.sqrt(d))
        check_grad(dq, r["dQ"], dtype, "dQ")
        for t, name in ((dk, "dK"), (dv, "dV")):
            check_grad(t[:, :, Tk - n:], r[name], dtype, name)
            assert not t[:, :, :Tk - n].any()
