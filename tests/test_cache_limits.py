"""Attention over a paged 8-bit cache at the limits of its arguments: value
scales that lie far apart or are no powers of two, ranges that end far below
zero, windows that decide how many blocks share a sequence; and appending with
positions and a scaled rotation.

Tolerances as test_cache.py's, row by row: bf16 rms 1e-2 of the row's, fp32
1e-5 of the row's sum of P |V| (which is what the roundings of weights and
scores go with), LSE 1e-4 and 1e-5 of its size.
"""
import math

import numpy as np
import pytest
import torch

import exact_tiled_softmax_attn_gb300 as B
from oracle import cache as ref
from oracle import scored as sref

from parity import check_o, np64
from test_cache import F8, as_oracle, attention_case, clean, i32, pool_of, table_of
from test_scored import check_lse


def compare(c, table, length, new, q, Tk, keys=None, **how):
    """forward_cached against the oracle, row by row; every row that sees a key has a result to be wrong in. keys: (K, V)
    where they are not what the pages hold."""
    dtype, scale = q.dtype, 1.0 / math.sqrt(q.shape[3])
    arrays = {n: None if how.get(n) is None else i32(how[n]) for n in ("q_pos", "key_begin", "key_end")}
    o, lse = B.forward_cached(q, c, table, i32(length), new_len=i32(new), Tk=Tk, causal=how.get("causal", True),
                              window=how.get("window", 0), **arrays)
    torch.cuda.synchronize()
    assert B.attn_device_status() == B.ATTN_OK
    k, v = keys or as_oracle(c, table, length, Tk)
    r = ref.attend(q, k, v, length, new, scale, **how)
    assert np.abs(r["O"]).max(-1)[np.isfinite(r["LSE"])].all()
    check_lse(lse, r["LSE"], dtype)
    with pytest.raises(AssertionError):   # (the bounds below would refuse zeros)
        check_o(np.zeros_like(r["O"]), r["O"], dtype)
    if dtype == torch.bfloat16:
        check_o(o, r["O"], dtype)
    else:
        size = ref.attend(q, k, np.abs(v), length, new, scale, **how)["O"].max(-1, keepdims=True)
        assert (np.abs(np64(o) - r["O"]) <= 1e-5 * size).all()
    return o, lse


def set_pages(c, table, b, scales, empty):
    """The value scales of sequence b's pages, in order; the codes of those in `empty` are all 0."""
    for i, s in enumerate(scales):
        at = int(table[b, i])
        c.v_scale[at] = s
        if empty[i]:
            c.v.view(torch.uint8)[at] = 0


SHAPES = [(16, 64, 64), (64, 128, 128), (128, 96, 128)]      # page, d, dv


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind", ["huge", "falling", "rising", "by turns"])
@pytest.mark.parametrize("page,d,dv", SHAPES)
@pytest.mark.parametrize("Tq", [1, 6, 13, 30, 60, 100])      # 2 to 200 rows a key head
def test_zeros_with_large_scales(Tq, page, d, dv, kind, dtype):
    """Pages of zeros whose scales are up to 2^64 times those of the pages that hold something: the scale of a page says
    nothing about the tokens that are seen."""
    shape = (2, 4, 2, Tq, 1300, d, dv, page)
    c, table, length, new, q = attention_case(shape, "e4m3", dtype, True, seed=3)
    n = table.shape[1]
    for b in range(2):
        i = np.arange(n)
        if kind == "huge":
            empty = i % 3 == 1
            scales = np.where(empty, 2.0 ** 40, 2.0 ** -8)
        elif kind == "by turns":
            empty = (i % 4 == 0) | (i % 4 == 3)
            scales = np.where(empty, 2.0 ** (10.0 * (i % 5)), 2.0 ** (-24.0 + i % 3))
        else:
            e = np.round(np.linspace(-24, 40, n))
            e = e[::-1] if kind == "falling" else e
            empty, scales = e > -16, 2.0 ** e
        set_pages(c, table, b, scales, empty)
    # (rows that see only pages of zeros have no result)
    compare(c, table, length, new, q, 1300, causal=False)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("page,d,dv", SHAPES)
@pytest.mark.parametrize("Tq", [1, 6, 13, 30, 60, 100])
def test_missing_pages_beside_small_scales(Tq, page, d, dv, dtype):
    """Table entries that name no page read as zeros, however small the other pages' values are."""
    shape = (2, 4, 2, Tq, 1300, d, dv, page)
    c, table, length, new, q = attention_case(shape, "e4m3", dtype, True, seed=5)
    c.v_scale.fill_(2.0 ** -35)
    table[0, 2], table[1, 0], table[1, 5] = -1, 1 << 30, c.k.shape[0]
    compare(c, table, length, new, q, 1300, causal=False)


@pytest.mark.gpu
@pytest.mark.parametrize("page,d,dv", SHAPES)
@pytest.mark.parametrize("last", [False, True])
@pytest.mark.parametrize("Tq", [1, 6, 13, 30, 60, 100])
def test_large_values_of_small_weight(Tq, page, d, dv, last):
    """A page whose keys have weights of 2^-50 and values 2^64 times the others' decides the result."""
    shape = (2, 4, 2, Tq, 1300, d, dv, page)
    c, table, length, new, q = attention_case(shape, "e4m3", torch.bfloat16, True, seed=7)
    # one sign of q and k, but for that page's keys: scores of about 17 and -17, 50 in units of log2 apart
    q = torch.full_like(q, 17.3 / math.sqrt(d))
    c.k.copy_(torch.ones(c.k.shape)), c.k_scale.fill_(1.0)
    n = table.shape[1]
    for b in range(2):
        at = n - 3 if last else 1
        scales = np.full(n, 2.0 ** -24)
        scales[at] = 2.0 ** 40
        set_pages(c, table, b, scales, np.zeros(n, bool))
        c.k[int(table[b, at])] = -c.k[int(table[b, at])].float()
    compare(c, table, length, new, q, 1300, causal=False)


@pytest.mark.gpu
@pytest.mark.parametrize("Tq", [1, 6, 16, 30, 60])
@pytest.mark.parametrize("Hkv", [1, 4])
def test_scales_far_apart_in_long_sequences(Hkv, Tq):
    """Sequences that the parts of many blocks are joined for, scales of any size per page and head, two pages in three
    of zeros."""
    shape = (3, 2 * Hkv, Hkv, Tq, 12000, 128, 128, 64)
    c, table, length, new, q = attention_case(shape, "e4m3", torch.bfloat16, True, seed=9)
    g = torch.Generator().manual_seed(1)
    e = torch.randint(-24, 41, c.v_scale.shape, generator=g).float()
    c.v_scale.copy_(torch.exp2(e))
    c.v.view(torch.uint8)[(e > -10).cuda()] = 0
    o, lse = compare(c, table, length, new, q, 12000)
    again = B.forward_cached(q, c, table, i32(length), new_len=i32(new), Tk=12000)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("Tq", [1, 6, 13, 30, 60, 100])
def test_ranges_that_end_far_below_zero(Tq, dtype):
    """A range's end may be any int32: one of -2^31 is an empty range, beside rows that see keys from every tile."""
    shape = (2, 4, 2, Tq, 700, 64, 64, 32)
    c, table, length, new, q = attention_case(shape, "e4m3", dtype, False, seed=11)
    end = np.full((2, Tq), 700)
    end[:, 1::3] = -2 ** 31
    end[:, 2::6] = -2 ** 31 + 100
    end[1, 0] = -2 ** 31
    compare(c, table, length, new, q, 700, causal=False, key_end=end)
    pos = np.where(end < 0, -2 ** 31, 650)
    compare(c, table, length, new, q, 700, q_pos=pos)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("page,d,dv", SHAPES)
@pytest.mark.parametrize("Tq", [1, 6, 13, 30, 60, 100])
def test_scales_that_are_no_powers_of_two(Tq, page, d, dv, dtype):
    """Scales of any size and any bits, and ones outside the range that scales are read in. The path that reads the
    pages into the workspace (more than 128 rows) rounds keys and values to the type: the oracle takes those."""
    shape = (2, 4, 2, Tq, 700, d, dv, page)
    c, table, length, new, q = attention_case(shape, "e4m3", dtype, True, seed=13)
    g = torch.Generator().manual_seed(3)
    c.k_scale.copy_(torch.exp2(torch.rand(c.k_scale.shape, generator=g) * 6 - 12))
    c.v_scale.copy_(torch.exp2(torch.rand(c.v_scale.shape, generator=g) * 60 - 30))
    c.v_scale[int(table[0, 2])], c.k_scale[int(table[0, 3])] = 0.0, 1e-30
    keys = None
    if 2 * Tq > 128 and dtype == torch.bfloat16:
        keys = [np64(x) for x in B.cache_read(c, table, i32(length), Tk=700)]
    compare(c, table, length, new, q, 700, keys=keys)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("store", ["e4m3", "plain"])
@pytest.mark.parametrize("Tq,window", [(1, 300), (4, 100), (6, 1000), (8, 300)])
def test_windows_in_long_sequences(Tq, window, store, dtype):
    """A window that leaves so few keys that blocks share them without a workspace, although the sequences' bound asks
    for one; with positions given, the bound decides."""
    shape = (3, 8, 2, Tq, 20000, 64, 64, 64)
    c, table, length, new, q = attention_case(shape, store, dtype, True, seed=15)
    length = [20000, 7001, 90]
    clean(c, table, length)
    code = B.ATTN_CACHE_E4M3 if store == "e4m3" else B.ATTN_CACHE_PLAIN
    size = B.attn_fwd_cached_workspace_size(3, 8, 2, Tq, 20000, 64, 64, code,
                                            B.ATTN_BF16 if dtype == torch.bfloat16 else B.ATTN_F32)
    assert size > 0
    compare(c, table, length, new, q, 20000, window=window)
    pos = np.array([[19990], [5000], [60]]) - 37 * np.arange(Tq)[None]
    compare(c, table, length, new, q, 20000, window=window, q_pos=np.maximum(pos, 0))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("store", ["e4m3", "plain"])
@pytest.mark.parametrize("mscale", [1.0, 1.3, 0.37])
@pytest.mark.parametrize("T,d,rot,inter,odd", [(1, 128, 128, False, 0), (3, 96, 64, True, 0), (70, 128, 64, False, 0),
                                               (130, 64, 64, True, 0), (40, 80, 40, False, 0), (70, 64, 64, False, 1)])
def test_append_with_positions_and_a_scaled_rotation(T, d, rot, inter, odd, mscale, store, dtype):
    """pos in place of the tokens' indexes, of any sign, and mscale in the keys, the queries and the scale's bound.
    Tolerances as test_cache.py's test_append, the rotation's times mscale."""
    Bn, H, Hkv, dv, page = 2, 4, 2, 64, 32
    store = F8 if store == "e4m3" else dtype
    g = torch.Generator().manual_seed(T + d)
    x = torch.randn(Bn, T, H * d + Hkv * (d + dv) + odd, generator=g).to(dtype).cuda()[:, :, odd:]
    q = x[..., :H * d].view(Bn, T, H, d).transpose(1, 2)
    k = x[..., H * d:(H + Hkv) * d].view(Bn, T, Hkv, d).transpose(1, 2)
    v = x[..., (H + Hkv) * d:].view(Bn, T, Hkv, dv).transpose(1, 2)
    held = [37, 0]
    seq_len, new = i32([h + T for h in held]), [T, T]
    per = (37 + T) // page + 1
    table = table_of(Bn, per, 1, 3)
    kp, ks = pool_of(Bn * per + 1, Hkv, page, d, store, 1)
    vp, vs = pool_of(Bn * per + 1, Hkv, page, dv, store, 2)
    c = B.KVCache(kp, vp, ks, vs)
    clean(c, table, i32(held))
    old, old_scale = np64(kp.float()), None if ks is None else np64(ks)
    pos = np.random.default_rng(T).integers(-2 ** 20, 2 ** 20, (Bn, T))
    got = B.cache_append(c, k, v, table, seq_len, plan=B.rope_plan(rot, interleaved=inter, mscale=mscale), q=q, pos=i32(pos))
    torch.cuda.synchronize()
    m = float(np.float32(mscale))
    freq = sref.rope_frequencies(rot)
    step = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24

    def near(a):     # |u| + |v| of the pair of every element (0 where nothing is turned)
        a = np.abs(np64(a))
        i = np.arange(rot)
        z = np.zeros_like(a)
        z[..., :rot] = a[..., i] + a[..., i ^ 1 if inter else (i + rot // 2) % rot]
        return z * m * 8 * 2.0 ** -24
    want = ref.rotated(q, pos, freq, inter, m)
    assert (np.abs(np64(got) - want) <= near(q) + step * np.abs(want)).all()
    kr = ref.rotated(k, pos, freq, inter, m)
    size = ref.key_size(np64(k), rot, m).astype(np.float32).max(-1)
    _, want_scale, fresh = ref.append(old, old_scale, table.cpu().numpy(), np64(seq_len), new, kr, size, page)
    exact, _, _ = ref.append(old, None, table.cpu().numpy(), np64(seq_len), new, kr, size, page)
    slack, _, _ = ref.append(old, None, table.cpu().numpy(), np64(seq_len), new, near(k), size, page)
    if ks is None:
        assert (np.abs(np64(kp) - exact) <= slack + step * np.abs(exact))[fresh].all()
    else:
        assert np.array_equal(np64(ks), want_scale)
        s = want_scale[:, :, None, None]
        off = np.abs(np64(kp.float()) * s - exact)
        assert (off <= slack + np.maximum(2.0 ** -4 * np.abs(exact), 2.0 ** -10 * s))[fresh].all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("page,d,dv", SHAPES)
@pytest.mark.parametrize("Tq", [1, 6, 13, 30, 60, 100])
def test_nan_beside_scales_far_apart(Tq, page, d, dv, dtype):
    """NaN behind the length changes nothing; a NaN in a value that rows see makes that element of their O NaN and leaves
    the others as they are."""
    shape = (2, 4, 2, Tq, 1290, d, dv, page)
    c, table, length, new, q = attention_case(shape, "e4m3", dtype, True, seed=17)
    n = table.shape[1]
    i = np.arange(n)
    for b in range(2):
        set_pages(c, table, b, np.where(i % 3 == 1, 2.0 ** 30, 2.0 ** -8), i % 3 == 1)
    how = dict(new_len=i32(new), Tk=1290, causal=False)
    o, lse = compare(c, table, length, new, q, 1290, causal=False)
    for b in range(2):
        for p in c[:2]:
            p.view(torch.uint8)[int(table[b, length[b] // page]), :, length[b] % page:] = 0x7f
    o2, lse2 = B.forward_cached(q, c, table, i32(length), **how)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    c.v.view(torch.uint8)[int(table[0, 0]), 1, 3, 7] = 0xff
    o3, lse3 = B.forward_cached(q, c, table, i32(length), **how)
    assert torch.isnan(o3[0, 2:, :new[0], 7]).all() and torch.equal(lse, lse3)
    o3[0, 2:, :, 7] = o[0, 2:, :, 7]
    assert torch.equal(o, o3)
    # in a page of zeros with a large scale too
    c.v.view(torch.uint8)[int(table[0, 1]), 1, 3, 9] = 0x7f
    o4, lse4 = B.forward_cached(q, c, table, i32(length), **how)
    assert torch.isnan(o4[0, 2:, :new[0], [7, 9]]).all() and torch.equal(lse, lse4)
    o4[0, 2:, :, 7], o4[0, 2:, :, 9] = o[0, 2:, :, 7], o[0, 2:, :, 9]
    assert torch.equal(o, o4)
