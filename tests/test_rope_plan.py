"""The plan of rotary positions against 60-digit arithmetic: every frequency is
the one of the formula, rounded to 2^-64 of a turn, so that a phase is off by at
most |pos| * 2^-65 turns before its upper 32 bits are taken."""
from decimal import Decimal, localcontext

import pytest
import torch

import exact_tiled_softmax_attn_gb300 as B

PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


def units(rot, theta=10000.0, factor=1.0, original_length=0.0, low_turns=1.0, high_turns=4.0, mscale=1.0):
    """f_i / (2 pi) * 2^64, of the doubles given."""
    theta, factor, length, low, high = (Decimal(x) for x in (theta, factor, original_length, low_turns, high_turns))
    out = []
    for i in range(rot // 2):
        turns = (theta.ln() * Decimal(-2 * i) / rot).exp() / (2 * PI)
        keep = Decimal(0)
        if length > 0:
            keep = min(max((length * turns - low) / (high - low), Decimal(0)), Decimal(1))
        out.append((turns * keep + turns / factor * (1 - keep)) * 2 ** 64)
    return out


@pytest.mark.parametrize("kw", [
    dict(rot=2), dict(rot=64), dict(rot=128), dict(rot=256), dict(rot=96, theta=500000.0), dict(rot=30, theta=1e300),
    dict(rot=254, theta=1.0000001), dict(rot=2, theta=1e308), dict(rot=96, factor=3.3), dict(rot=128, factor=1e12),
    dict(rot=256, theta=500000.0, factor=8.0, original_length=8192.0, low_turns=1.0, high_turns=32.0),
    dict(rot=128, factor=40.0, original_length=4096.0, low_turns=0.1, high_turns=0.7)])
def test_frequencies_are_the_formulas(kw):
    p = B.rope_plan(**kw)
    with localcontext() as c:
        c.prec = 60
        off = [abs(int(p.turns[i]) - u) for i, u in enumerate(units(**kw))]
    # half a unit, and what some 100 bits of the intermediate values leave
    assert max(off) <= Decimal(0.5) + Decimal(2) ** -30


@pytest.mark.gpu
def test_phases_at_the_ends_of_int32():
    """cos and sin of exact phases (Python integers) at positions up to +-2^31."""
    rot = 64
    plan = B.rope_plan(rot, theta=10000.0)
    pos = torch.tensor([[-2 ** 31, 2 ** 31 - 1, 2 ** 30 + 12345, -987654321, 7, 0]], dtype=torch.int32)
    x = torch.zeros(1, 1, 6, rot, device="cuda")
    x[..., :rot // 2] = 1.0                      # (u, v) = (1, 0): the results are cos and sin
    y, _ = B.rope(x, x, plan, pos=pos.cuda())
    with localcontext() as c:
        c.prec = 60
        f = units(rot, theta=10000.0)
        turns = [[float(int(p) * u / 2 ** 64 % 1) for u in f] for p in pos[0].tolist()]
    a = torch.tensor(turns, dtype=torch.float64) * 2 * float(PI)
    want = torch.cat((a.cos(), a.sin()), -1)
    # 2^-34 turns from the frequency and 2^-32 from the phase's upper bits (1.9e-9 radians), then a few 2^-24
    assert (y[0, 0].cpu().double() - want).abs().max() <= 4 * 2.0 ** -24
