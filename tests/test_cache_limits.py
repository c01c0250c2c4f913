"""Attention over a paged 8-bit cache at the limits of its arguments: value
scales that lie far apart, ranges that end far below zero.

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

from parity import check_o, np64
from test_cache import as_oracle, attention_case, i32
from test_scored import check_lse


def compare(c, table, length, new, q, Tk, **how):
    """forward_cached against the oracle, row by row; every row that sees a key has a result to be wrong in."""
    dtype, scale = q.dtype, 1.0 / math.sqrt(q.shape[3])
    arrays = {n: None if how.get(n) is None else i32(how[n]) for n in ("q_pos", "key_begin", "key_end")}
    o, lse = B.forward_cached(q, c, table, i32(length), new_len=i32(new), Tk=Tk, causal=how.get("causal", True),
                              window=how.get("window", 0), **arrays)
    torch.cuda.synchronize()
    assert B.attn_device_status() == B.ATTN_OK
    k, v = as_oracle(c, table, length, Tk)
    r = ref.attend(q, k, v, length, new, scale, **how)
    assert np.abs(r["O"]).max(-1)[np.isfinite(r["LSE"])].all()
    check_lse(lse, r["LSE"], dtype)
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
