"""Which calls of attn_rope are refused for an overlap: none but those in which
a row of an output shares a byte with another row of it, with the other output,
an input or the positions."""
import ctypes
import itertools
import os
import random
import shutil
import subprocess

import pytest
import torch

import exact_tiled_softmax_attn_gb300 as B

from test_rope import _rope

CSRC = os.path.join(os.path.dirname(os.path.abspath(B.__file__)), "csrc")


@pytest.fixture(scope="module")
def views(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("needs g++")
    where = tmp_path_factory.mktemp("views")
    (where / "v.cc").write_text('''
#include "views.h"
using namespace attn;
static Rows rows(const long long* x) { return Rows{(uintptr_t)x[0], x[1], {x[2], x[3], x[4]}, {x[5], x[6], x[7]}}; }
extern "C" int distinct_(const long long* a) { return distinct(rows(a)); }
extern "C" int apart_(const long long* a, const long long* b) { return apart(rows(a), rows(b)); }
''')
    subprocess.run([gxx, "-O1", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, "-o", str(where / "v.so"),
                    str(where / "v.cc")], check=True)
    lib = ctypes.CDLL(str(where / "v.so"))
    pack = lambda r: (ctypes.c_longlong * 8)(r[0], r[1], *r[2], *r[3])  # noqa: E731
    return (lambda a: bool(lib.distinct_(pack(a)))), (lambda a, b: bool(lib.apart_(pack(a), pack(b))))


def starts(r):
    base, _, step, n = r
    return [base + sum(i * s for i, s in zip(at, step)) for at in itertools.product(*(range(k) for k in n))]


def test_views_against_every_byte(views):
    """Small views of random steps, orders and offsets: the answers are those of marking every byte."""
    distinct, apart = views
    g = random.Random(1)
    seen = {True: 0, False: 0}
    for _ in range(6000):
        def one():
            n = [g.randint(1, 4) for _ in range(3)]
            w = g.randint(1, 6)
            step = [g.choice([g.randint(0, 60), 8, 16, 24, 48]) for _ in range(3)]
            return g.randint(0, 120), w, step, n
        a, b = one(), one()
        bytes_of = lambda r: [x + i for x in starts(r) for i in range(r[1])]  # noqa: E731
        x, y = bytes_of(a), bytes_of(b)
        assert distinct(a) == (len(set(x)) == len(x)), a
        assert apart(a, b) == (not set(x) & set(y)), (a, b)
        seen[apart(a, b)] += 1
    assert min(seen.values()) > 500


def test_views_of_one_buffer(views):
    """Queries and keys in one buffer of every order of its dimensions, at the sizes of real calls."""
    _, apart = views
    Bn, T, H, d = 7, 65521, 24, 256
    for order in itertools.permutations("bt3h"):
        size = dict(b=Bn, t=T, h=H)
        size["3"] = 3
        step, at = {}, d
        for c in reversed(order):
            step[c] = at
            at *= size[c]
        q = (0, d, [step["b"], step["h"], step["t"]], [Bn, H, T])
        k = (step["3"], *q[1:])
        assert apart(q, k) and apart(k, q)
        assert not apart(q, (step["3"] - 1, *q[1:])) or step["3"] != d
        assert not apart(q, (step["t"], *q[1:]))


@pytest.mark.parametrize("kw", [
    dict(Kout=0x300000, Qout=0x300000 + 2 * 1024),                   # over the second half of the keys
    dict(Q=0x100000, Qout=0x100000, strides=[4096, 512, 64, 4096, 64, 512] + [2048, 512, 64] * 2),   # transposed
    dict(pos=0x200000 + 2 * 64 * 63),                                # inside the last row of an output
])
def test_overlaps_are_refused(kw):
    assert _rope(**kw) == B.ATTN_ERR_INVALID_ARG


LAYOUTS = ["3bhtd", "b3htd", "bth3d", "tb3hd", "bh3td", "htb3d", "t3bhd"]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_in_place_in_a_fused_projection_of_any_layout(layout, dtype):
    size = dict(b=3, t=19, h=4, d=64)
    size["3"] = 3
    g = torch.Generator().manual_seed(3)
    buf = torch.randn(*(size[c] for c in layout), generator=g).to(dtype).cuda()
    view = buf.permute(*(layout.index(c) for c in "3bhtd"))
    keep = view.clone()
    q, k, v = view
    plan = B.rope_plan(64)
    want = B.rope(q.contiguous(), k.contiguous(), plan)
    out = B.rope(q, k, plan, out=(q, k))
    assert out[0] is q and out[1] is k
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, keep[2])
    # and from one part of it to another
    view.copy_(keep)
    B.rope(q, v, plan, out=(q, k))
    want = B.rope(keep[0], keep[2], plan)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, keep[2])
