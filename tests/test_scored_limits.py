"""Scored attention at the ends of what it accepts: caps far above the scores.

Tolerances are those of the other bf16 tests of the scored attention: with a
cap of any size a score is off by a few 2^-24 of itself, below 1e-4 for the
scores of these inputs (up to 50).
"""
import math
import os
import re
import types

import numpy as np
import pytest
import torch

import exact_tiled_softmax_attn_gb300 as B
from exact_tiled_softmax_attn_gb300 import binding
from oracle import scored as ref

from parity import check_o, frob_rel, np64
from test_scored import check_grad, check_lse, how_of, magnitudes, make, run_case

CSRC = os.path.join(os.path.dirname(os.path.abspath(B.__file__)), "csrc")


# ------------------------------------------------------------------ the cap

def relative_fit(degree, top):
    """The polynomial of tanh(x) / x in x^2 on (0, top] with the least largest relative error: (error, coefficients).

    Least squares, reweighted by the errors until the largest are equal (Lawson)."""
    x = top * np.sin(np.linspace(0.0, np.pi / 2, 4001))[1:]
    want = np.tanh(x) / x
    a = np.vander((x / top) ** 2, degree + 1, increasing=True)
    w = np.full(len(x), 1.0 / len(x))
    best = (1.0, None)
    for _ in range(400):
        s = np.sqrt(w) / want
        c = np.linalg.lstsq(a * s[:, None], want * s, rcond=None)[0]
        e = np.abs(a @ c / want - 1.0)
        if e.max() < best[0]:
            best = (e.max(), c / top ** (2 * np.arange(degree + 1)))
        w = w * e
        w /= w.sum()
    return best


@pytest.mark.parametrize("degree,top,bound", [(2, 0.25, 4.0e-7), (4, 0.6, 7.4e-8)])
def test_the_caps_polynomials_are_their_fits(degree, top, bound):
    text = open(os.path.join(CSRC, "scored_math.cuh")).read()
    assert "kCapLimit%d = %gf" % (degree, top) in text
    held = [float(t) for t in re.search(r"kCapPoly%dFit\[%d\] = \{([^}]*)\}" % (degree, degree + 1),
                                        text).group(1).split(",")]
    x = np.linspace(0.0, top, 20001)[1:]
    assert np.abs(np.polyval(held[::-1], x * x) * x / np.tanh(x) - 1.0).max() <= bound
    best, c = relative_fit(degree, top)
    assert best <= bound <= 1.02 * best
    assert np.abs(np.polyval((np.array(held) - c)[::-1], x * x)).max() <= 1e-9


CAPS = [(1e3, None), (5.5e3, None), (1e4, None), (1e5, None), (1e6, None), (50.0, 1.0 / 128), (1e6, 1.0 / 128),
        (1e-4, None), (3.0, 40.0)]


@pytest.mark.gpu
@pytest.mark.parametrize("cap,scale", CAPS)
@pytest.mark.parametrize("shape,mask,bias", [((1, 4, 2, 300, 300, 128, 128), "causal", False),
                                             ((2, 4, 4, 260, 300, 64, 64), "docs", True),
                                             ((1, 8, 1, 300, 260, 64, 64), "wild", False)])
def test_caps_of_any_size(shape, mask, bias, cap, scale):
    if scale != 40.0:
        run_case(shape, mask, cap, bias, torch.bfloat16, grad=True, scale=scale)
        return
    # Scores of a spread of 200 caps: T = 1 - (t / cap)^2 leaves a row two or three of its keys, and where those have
    # most of its weight, dP - D is small beside D. The O in D is rounded, by half a step of each element, so dS is off
    # by up to P T 2^-8 |dO| |O|, however small dP - D is: no bound in the norm of dQ, which T makes small too. The
    # bound by terms instead: dS rounded and D's O rounded (2 half steps of P (|dO| |V| + |dO| |O|)), for dK P T too,
    # and the result; T and P off by what the score is off, d roundings of its product, over the cap.
    run_case(shape, mask, cap, bias, torch.bfloat16, grad=False, scale=scale)
    Bn, H, Hkv, Tq, Tk, d, dv = shape
    x, how = make(*shape, torch.bfloat16, seed=Tq + 3 * Tk + d), how_of(mask, cap, bias, Bn, H, Tq, Tk)
    o, lse = B.forward_scored(*x[:3], scale=scale, **how)
    g = B.backward_scored(*x[:3], o, lse, x[3], scale=scale, **how)
    flat = dict(how, slopes=torch.zeros(H)) if how["slopes"] is None else how
    r, size = ref.scored(*x, scale=scale, **how), magnitudes(x, flat, scale)
    rel = 3 * 2.0 ** -8 + 2 * d * 2.0 ** -24 * size["score"] / cap + 1e-5
    for t, name in zip(g, ("dQ", "dK", "dV")):
        assert (np.abs(np64(t) - r[name]) <= rel * size[name] + 2.0 ** -8 * np.abs(r[name]) + 1e-6).all(), name


@pytest.mark.gpu
@pytest.mark.parametrize("cap,scale", CAPS)
@pytest.mark.parametrize("shape,mask,bias", [((1, 8, 8, 1, 3000, 128, 128), "causal", False),
                                             ((3, 16, 2, 2, 700, 64, 64), "window", True),
                                             ((2, 4, 1, 7, 300, 128, 64), "wild", False)])
def test_caps_of_any_size_with_few_rows(shape, mask, bias, cap, scale):
    run_case(shape, mask, cap, bias, torch.bfloat16, grad=False, scale=scale)


@pytest.mark.gpu
@pytest.mark.parametrize("cap", [30.0, 1e3, 1e5, 1e6])
@pytest.mark.parametrize("Tq", [5, 200])
def test_a_rows_scores_do_not_suffer_from_its_neighbours(Tq, cap):
    """One row's scores reach the cap, and so would those of keys that no row sees; the other rows' stay small."""
    Bn, H, Hkv, Tk, d = 1, 2, 2, 500, 64
    x = make(Bn, H, Hkv, Tq, Tk, d, d, torch.bfloat16, 61)
    x[0][:, :, 3] *= cap / 8
    x[1][:, :, Tk - 40:] *= cap / 8
    how = dict(softcap=cap, key_end=torch.full((Bn, Tq), Tk - 40, dtype=torch.int32, device="cuda"))
    o, lse = B.forward_scored(*x[:3], **how)
    dq, dk, dv = B.backward_scored(*x[:3], o, lse, x[3], **how)
    assert B.attn_device_status() == B.ATTN_OK
    r = ref.scored(*x, scale=1.0 / math.sqrt(d), **how)
    check_o(o, r["O"], torch.bfloat16)
    rest = [i for i in range(Tq) if i != 3]
    check_lse(lse[:, :, rest], r["LSE"][:, :, rest], torch.bfloat16)
    # beyond 0.6 of the cap: 3e-7 of the cap from the formula, and the sum of products' own rounding
    assert np.abs(np64(lse)[:, :, 3] - r["LSE"][:, :, 3]).max() <= 1e-4 + 2e-6 * cap
    check_grad(dq[:, :, rest], r["dQ"][:, :, rest], torch.bfloat16, "dQ")
    check_grad(dv, r["dV"], torch.bfloat16, "dV")
    assert not dk[:, :, Tk - 40:].any() and not dv[:, :, Tk - 40:].any()


# ------------------------------------------------------------------ rows and keys that nothing concerns

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (4.0, True)])
@pytest.mark.parametrize("shape", [(1, 2, 2, 3, 300, 64, 64), (1, 8, 1, 4, 2000, 128, 40), (2, 4, 2, 150, 300, 128, 64),
                                   (1, 1, 1, 300, 2100, 64, 64), (1, 8, 1, 300, 260, 64, 64)])
def test_zeros_beside_infinities_that_others_see(shape, cap, bias, dtype):
    """Rows that see no key give O = 0, LSE = -inf and dQ = 0, and keys before and behind every range dK = dV = 0,
    whatever the rows and keys of others hold: infinite V and K in their ranges, NaN in their dO."""
    Bn, H, Hkv, Tq, Tk, d, dv = shape
    x = make(*shape, dtype, 67)
    how = how_of("none", cap, bias, Bn, H, Tq, Tk)
    empty = torch.arange(Tq) % 3 == 1
    how["key_begin"] = torch.full((Bn, Tq), 2, dtype=torch.int32, device="cuda")
    how["key_end"] = torch.where(empty, 0, Tk - 3).to(torch.int32).expand(Bn, Tq).contiguous().cuda()
    at = empty.nonzero()[:, 0].cuda()

    def check():
        o, lse = B.forward_scored(*x[:3], **how)
        assert not o[:, :, at].any() and torch.isneginf(lse[:, :, at]).all()
        dq, dk, dv_ = B.backward_scored(*x[:3], o, lse, x[3], **how)
        assert B.attn_device_status() == B.ATTN_OK
        assert not dq[:, :, at].any()
        for t in (dk, dv_):
            assert not t[:, :, :2].any() and not t[:, :, Tk - 3:].any()
    check()
    x[2][:, :, Tk // 2] = float("inf")
    check()
    x[3][:, :, 0] = float("nan")
    check()
    x[1][:, :, 5] = float("inf")
    check()


# ------------------------------------------------------------------ what a row does see

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 2, 2, 1, 3000, 64, 64), (1, 8, 1, 4, 2000, 128, 40), (2, 4, 2, 150, 300, 128, 64),
                                   (1, 2, 1, 300, 3000, 64, 64)])
def test_a_nan_among_the_values_shows_whatever_its_weight(shape, dtype):
    """A steep bias leaves far keys weights below fp32's range, in ranges of keys of their own too; a NaN in one
    element of such a key's value is a NaN in that column of O, and nowhere else."""
    Bn, H, Hkv, Tq, Tk, d, dv = shape
    x = make(*shape, dtype, 71, grad=False)
    how = dict(slopes=torch.full((H,), 2.0, device="cuda"),
               q_pos=torch.full((Bn, Tq), Tk, dtype=torch.int32, device="cuda"))
    want = B.forward_scored(*x, **how)
    x[2][:, :, 17, 3] = float("nan")
    o, lse = B.forward_scored(*x, **how)
    assert B.attn_device_status() == B.ATTN_OK
    assert o[..., 3].isnan().all()
    o[..., 3] = want[0][..., 3]
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


# ------------------------------------------------------------------ what is handed in beside the inputs

@pytest.mark.parametrize("workspace", [torch.zeros(1 << 20), torch.zeros(1, dtype=torch.uint8).expand(1 << 20),
                                       torch.zeros(1 << 21, dtype=torch.uint8)[::2]], ids=["f32", "repeated", "strided"])
def test_a_workspace_of_another_kind_is_refused(workspace):
    q, k = torch.zeros(1, 4, 8, 64), torch.zeros(1, 2, 8, 64)
    with pytest.raises(ValueError, match="workspace"):
        B.forward_scored(q, k, k, workspace=workspace)
    with pytest.raises(ValueError, match="workspace"):
        B.backward_scored(q, k, k, q, q[..., 0].contiguous(), q, workspace=workspace)


@pytest.mark.gpu
def test_a_workspace_of_the_host_is_refused_and_one_of_the_device_serves():
    x = make(1, 4, 2, 300, 300, 64, 64, torch.bfloat16, 73)
    n = [f(1, 4, 2, 300, 300, 64, 64, B.ATTN_BF16) for f in (B.attn_fwd_scored_workspace_size,
                                                            B.attn_bwd_scored_workspace_size)]
    with pytest.raises(ValueError, match="workspace"):
        B.forward_scored(*x[:3], workspace=torch.zeros(n[0], dtype=torch.uint8))
    o, lse = B.forward_scored(*x[:3], workspace=torch.empty(n[0], dtype=torch.uint8, device="cuda"))
    ws = torch.empty(n[1], dtype=torch.uint8, device="cuda")
    g = B.backward_scored(*x[:3], o, lse, x[3], workspace=ws)
    want = B.forward_scored(*x[:3])
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert all(torch.equal(a, b) for a, b in zip(g, B.backward_scored(*x[:3], *want, x[3])))
    with pytest.raises(B.AttnError):
        B.backward_scored(*x[:3], o, lse, x[3], workspace=ws[:-1])


def test_a_stream_of_another_device_is_refused():
    """Before anything is made current or launched: the kernels would run on the stream's device."""
    def call(*a):
        raise AssertionError("called")
    other = types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0)
    with pytest.raises(ValueError, match="stream"):
        binding._call_on(0, other, call)


@pytest.mark.gpu
def test_streams_of_the_tensors_device_serve():
    x = make(1, 4, 2, 70, 90, 64, 64, torch.bfloat16, 79, grad=False)
    want = B.forward_scored(*x)
    torch.cuda.synchronize()
    for s in (torch.cuda.Stream(), torch.cuda.default_stream(), torch.cuda.current_stream()):
        o, lse = B.forward_scored(*x, stream=s)
        s.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


# ------------------------------------------------------------------ how often a gradient is rounded

@pytest.mark.gpu
@pytest.mark.parametrize("cap", [0.0, 8.0])
@pytest.mark.parametrize("H,Hkv,T", [(2, 2, 700), (8, 1, 400)])   # (the second in parts of row tiles)
def test_roundings_of_the_gradients(H, Hkv, T, cap):
    """dQ and dK: dS and the result are rounded to bf16, and the O in D is; dV: P and the result. Nothing else.

    A rounding to bf16 moves a tensor of these gradients by r = 0.00166 of its norm (measured on the results, in
    float64); roundings of independent terms of a sum of independent terms move the sum by as much; independent errors
    add in squares. What the rounded O does to D is formed from the formula. One rounding more would be at least a
    sixth more."""
    d = 128
    x = make(1, H, Hkv, T, T, d, d, torch.bfloat16, 83)
    o, lse = B.forward_scored(*x[:3], causal=True, softcap=cap)
    g = B.backward_scored(*x[:3], o, lse, x[3], causal=True, softcap=cap)
    how = dict(scale=1.0 / math.sqrt(d), causal=True, softcap=cap)
    r = ref.scored(*x, **how)
    # the formula with the rounded O in D: D enters dS linearly, so its error's share is that of dO o (O - O')
    q, k, _, do = (np64(t)[0] for t in x)
    extra = (do * (np64(o)[0] - r["O"][0])).sum(-1)
    dq, dk = np.zeros_like(q), np.zeros_like(k)
    for h in range(H):
        s = how["scale"] * q[h] @ k[h * Hkv // H].T
        t = 1.0
        if cap:
            s = cap * np.tanh(s / cap)
            t = 1.0 - (s / cap) ** 2
        p = np.where(np.tri(T, dtype=bool), np.exp(s - r["LSE"][0, h][:, None]), 0.0)
        ds = -p * extra[h][:, None] * t * how["scale"]
        dq[h] = ds @ k[h * Hkv // H]
        dk[h * Hkv // H] += ds.T @ q[h]
    for t, name, off in zip(g, ("dQ", "dK", "dV"), (dq, dk, 0.0)):
        want = r[name]
        once = frob_rel(torch.from_numpy(want).to(torch.bfloat16), want)
        assert 0.0015 < once < 0.0018
        bound = math.sqrt(2 * once ** 2 + (np.linalg.norm(off) / np.linalg.norm(want)) ** 2)
        err = frob_rel(t, want)
        assert err <= 1.08 * bound, (name, err, bound)


# ------------------------------------------------------------------ rows whose weight lies on a few keys

FEW = [  # B, H, Hkv, Tq, Tk, d, dv
    ((1, 5, 1, 54, 2, 40, 64), "window", 0.5, True),
    ((2, 2, 1, 59, 3, 40, 8), "window", 0.0, True),
    ((1, 15, 3, 4, 4, 8, 80), "docs", 0.0, True),
    ((3, 9, 3, 330, 2, 128, 8), "prefix", 0.0, False),
    ((1, 3, 1, 7, 3, 72, 128), "causal", 700.0, False),
    ((2, 6, 2, 24, 2, 16, 80), "causal", 1e5, False),
    ((2, 4, 2, 574, 2, 64, 64), "wild", 1e5, False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("shape,mask,cap,bias", FEW)
def test_gradients_of_rows_that_see_few_keys(shape, mask, cap, bias):
    """dP - D is small beside D there: a D formed from the rounded O alone put dQ off by up to 0.02 of its norm."""
    run_case(shape, mask, cap, bias, torch.bfloat16, grad=True)


def short_documents(T, longest, seed):
    g = np.random.default_rng(seed)
    edge = [0]
    while edge[-1] < T:
        edge.append(min(T, edge[-1] + int(g.integers(2, longest + 1))))
    begin = np.concatenate([np.full(b - a, a) for a, b in zip(edge, edge[1:])])
    return begin.astype(np.int32)[None], np.concatenate([np.full(b - a, b) for a, b in zip(edge, edge[1:])]).astype(np.int32)[None]


@pytest.mark.gpu
@pytest.mark.parametrize("longest", [3, 12, 60])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (8.0, False), (0.0, True), (8.0, True)])
@pytest.mark.parametrize("H,Hkv,d", [(4, 2, 64), (2, 2, 128)])
def test_gradients_over_short_documents_are_rounded_twice(H, Hkv, d, cap, bias, longest):
    """dS and the result are rounded to bf16, nothing else: sqrt(2) of what rounding the exact gradients is (see
    test_roundings_of_the_gradients), and a tenth for what is left of the rounding of O in D (a fifth of it at most,
    where P goes into its correction in 11 bits) and for the spread of a few hundred rows."""
    T = 700
    x = make(1, H, Hkv, T, T, d, d, torch.bfloat16, 89)
    begin, end = short_documents(T, longest, 90)
    how = dict(softcap=cap, key_begin=torch.from_numpy(begin).cuda(), key_end=torch.from_numpy(end).cuda(),
               slopes=torch.exp2(-torch.arange(1.0, H + 1)).cuda() if bias else None)
    o, lse = B.forward_scored(*x[:3], **how)
    g = B.backward_scored(*x[:3], o, lse, x[3], **how)
    assert B.attn_device_status() == B.ATTN_OK
    r = ref.scored(*x, scale=1.0 / math.sqrt(d), **how)
    for t, name in zip(g, ("dQ", "dK", "dV")):
        once = frob_rel(torch.from_numpy(r[name]).to(torch.bfloat16), r[name])
        assert frob_rel(t, r[name]) <= 1.1 * math.sqrt(2) * once, name


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (6.0, True)])
def test_the_backward_on_parts_of_the_keys(cap, bias, dtype):
    """With O and LSE of all keys, the gradients of the keys' parts are the formula's: dQ in two shares, dK and dV by
    rows. (D is not the sum of P dP over a part.)"""
    Bn, H, Hkv, Tq, Tk, d = 1, 4, 2, 300, 560, 64
    x = make(Bn, H, Hkv, Tq, Tk, d, d, dtype, 97)
    how = how_of("none", cap, bias, Bn, H, Tq, Tk)
    o, lse = B.forward_scored(*x[:3], **how)
    r = ref.scored(*x, scale=1.0 / math.sqrt(d), **how)
    cut, dq = 250, 0.0
    for a, b in ((0, cut), (cut, Tk)):
        part = dict(how, q_pos=how["q_pos"] - a)
        k, v = (t[:, :, a:b].contiguous() for t in x[1:3])
        g = B.backward_scored(x[0], k, v, o, lse, x[3], **part)
        dq = dq + g[0].double()
        check_grad(g[1], r["dK"][:, :, a:b], dtype, "dK")
        check_grad(g[2], r["dV"][:, :, a:b], dtype, "dV")
    check_grad(dq, r["dQ"], dtype, "dQ")
