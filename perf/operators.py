"""Cases of the scored attention and rotary-position operators.

Two operators, as a language model's attention layer uses them one after the
other:

* rotary positions of queries and keys, and their transpose (the gradient);
* softmax attention whose scores are capped by a tanh, get a bias that falls
  with distance, and are limited to one range of keys per query row (causal,
  documents packed into one sequence, a prefix that every row sees, a sliding
  window), with query heads that share key heads: for prompts, for a training
  step (forward and backward), and for single tokens against a long cache.

`own` chooses between the plain form in elementary torch operations and the
calls of exact_tiled_softmax_attn_gb300.
"""
import math
import random

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ cases

def _rope(name, **kw):
    c = dict(op="rope", B=1, T=1, H=16, Hkv=16, d=128, rot=128, interleaved=False, inverse=False, far=8192,
             factor=1.0, parts=False, token_major=True, dtype="bf16")
    c.update(kw)
    return dict(c, name=name) if name else c


def _attn(name, op, **kw):
    c = dict(op=op, B=1, H=16, Hkv=16, Tq=128, Tk=128, d=128, dv=128, mask="causal", span=0, cap=0.0, bias=False,
             idle=False, dtype="bf16")
    c.update(kw)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one new token for each of 64 served sequences, at far positions: latency counts
        _rope("rope_tokens", B=64, T=1, H=16, Hkv=4, far=131072, factor=8.0, parts=True),
        # the queries and keys of a long prompt batch, taken from a [B, T, H, d] projection
        _rope("rope_prompt", B=2, T=8192, H=16, Hkv=16, far=8192),
        # gradient of an interleaved partial rotation in fp32, odd sizes
        _rope("rope_grad", B=3, T=1111, H=12, Hkv=4, d=96, rot=64, interleaved=True, inverse=True, far=5000,
              factor=4.0, dtype="f32"),
        # one sequence's next token, capped scores: the smallest call of the attention
        _attn("token_one", "tokens", B=1, H=8, Hkv=8, Tq=1, Tk=4096, cap=50.0),
        # the next token of 32 served sequences of all lengths, long caches, shared key heads
        _attn("tokens_long", "tokens", B=32, H=32, Hkv=8, Tq=1, Tk=32768, cap=30.0),
        # three tokens a sequence in a sliding window with a distance bias; some slots are idle
        _attn("tokens_window", "tokens", B=48, H=16, Hkv=2, Tq=3, Tk=9001, d=64, dv=64, mask="window", span=1024,
              bias=True, idle=True),
        # a prompt batch of documents packed into one sequence, shared key heads
        _attn("prompt_docs", "prompt", H=32, Hkv=8, Tq=8192, Tk=8192, mask="docs", span=1000),
        # the last part of a prompt against what the cache holds already, prefix visible to all, distance bias
        _attn("prompt_prefix", "prompt", B=2, H=16, Hkv=4, Tq=2047, Tk=5001, d=64, dv=64, mask="prefix", span=700,
              bias=True),
        # training step, capped scores, causal
        _attn("train_cap", "train", B=2, H=16, Hkv=16, Tq=4096, Tk=4096, cap=50.0),
        # training step on packed documents, shared key heads
        _attn("train_docs", "train", H=32, Hkv=8, Tq=8192, Tk=8192, mask="docs", span=1500),
        # training step with the distance bias, d = 64
        _attn("train_bias", "train", B=4, H=16, Hkv=16, Tq=2048, Tk=2048, d=64, dv=64, bias=True),
        # fp32 training step: cap, bias, documents and padding rows that see nothing
        _attn("train_f32", "train", B=2, H=8, Hkv=4, Tq=1000, Tk=1000, d=64, dv=64, mask="docs", span=300, cap=20.0,
              bias=True, idle=True, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "tokens", "prompt", "train"])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    H = Hkv * rng.choice([1, 1, 2, 4, 7, 8])
    if op == "rope":
        d = rng.choice([64, 80, 96, 128, 256])
        rot = rng.choice([d, d, d // 2, 32])
        B = _log(rng, 1, 64)
        T = _log(rng, 1, max(1, min(16384, 33000000 // (B * H * d))))
        return _rope(None, B=B, T=T, H=H, Hkv=Hkv, d=d, rot=rot, interleaved=rng.random() < 0.5,
                     inverse=rng.random() < 0.5, far=_log(rng, max(T, 64), 1000000),
                     factor=rng.choice([1.0, 2.0, 8.0, 32.0]), parts=rng.random() < 0.5,
                     token_major=rng.random() < 0.7, dtype=rng.choice(["bf16", "bf16", "f32"]))
    mods = dict(cap=rng.choice([0.0, 0.0, 15.0, 30.0, 50.0]), bias=rng.random() < 0.4, idle=rng.random() < 0.3)
    d = rng.choice([64, 64, 128, 128, 128, 80, 96, 40])
    dv = rng.choice([d, d, d, 64, 128])
    if op == "tokens":
        B = _log(rng, 1, 64)
        Tq = rng.choice([1, 1, 1, 2, 3, 5])
        Tk = _log(rng, 16, max(16, min(65536, 4200000 // (B * Hkv))))
        return _attn(None, op, B=B, H=H, Hkv=Hkv, Tq=Tq, Tk=Tk, d=d, dv=dv, mask=rng.choice(["causal", "window"]),
                     span=_log(rng, 16, 4096), dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]), **mods)
    dtype = rng.choice(["bf16", "bf16", "bf16", "bf16", "f32"])
    B = rng.choice([1, 1, 2, 3, 4])
    most = int(math.sqrt((1.6e7 if dtype == "f32" else 5e8) / (B * H)))
    Tk = _log(rng, 17, min(8192, most))
    mask = rng.choice(["none", "causal", "docs", "prefix", "window"])
    Tq = Tk if op == "train" or mask == "docs" or rng.random() < 0.4 else _log(rng, 1, Tk)
    return _attn(None, op, B=B, H=H, Hkv=Hkv, Tq=Tq, Tk=Tk, d=d, dv=dv, mask=mask,
                 span=_log(rng, 16, max(32, Tk // 2)), dtype=dtype, **mods)


# ------------------------------------------------------------------ what the cases hold

def _lengths(c):
    """Keys that each sequence of a token case has in its cache (its own new tokens among them)."""
    r = random.Random("%d %d %d" % (c["B"], c["Tk"], c["H"]))
    n = [max(c["Tq"], int(c["Tk"] * (0.15 + 0.85 * r.random()))) for _ in range(c["B"])]
    n[0] = c["Tk"]
    return [min(x, c["Tk"]) for x in n]


def _ranges(c):
    """numpy (key_begin, key_end, q_pos), each [B, Tq] or None, of an attention case."""
    B, Tq, Tk, mask = c["B"], c["Tq"], c["Tk"], c["mask"]
    i = np.arange(Tq)[None, :] + np.zeros((B, 1), np.int64)
    begin = end = None
    if c["op"] == "tokens":
        pos = np.asarray(_lengths(c))[:, None] - Tq + i
    else:
        pos = i + (Tk - Tq)
    if mask == "window":
        begin = np.maximum(pos - c["span"] + 1, 0)
    if mask == "docs":
        r = random.Random("%d %d %d" % (B, Tk, c["span"]))
        begin, end = np.zeros((B, Tq), np.int64), np.zeros((B, Tq), np.int64)
        for b in range(B):
            at = 0
            while at < Tk:
                n = max(1, int(c["span"] * math.exp(r.uniform(-1.2, 0.8))))
                to = min(Tk, at + n)
                begin[b, at:to], end[b, at:to] = at, to
                at = to
        end = np.minimum(end, pos + 1)
    elif mask == "prefix":
        end = np.maximum(pos + 1, np.minimum(c["span"], Tk))
    elif mask != "none":
        end = pos + 1
    if c["idle"]:
        begin = np.zeros((B, Tq), np.int64) if begin is None else begin.copy()
        end = np.full((B, Tq), Tk, np.int64) if end is None else end.copy()
        if c["op"] == "tokens":
            begin[B // 2:B // 2 + 1], end[B // 2:B // 2 + 1] = 0, 0   # a slot that serves nobody
        else:
            begin[:, Tq - Tq // 9:], end[:, Tq - Tq // 9:] = 0, 0     # padding rows behind the last token
    return begin, end, pos


def _pairs(c):
    """(allowed query-key pairs of one head summed over the batch, keys that some row of their sequence sees)."""
    begin, end, pos = _ranges(c)
    lo = np.zeros_like(pos) if begin is None else begin
    hi = np.full_like(pos, c["Tk"]) if end is None else np.minimum(end, c["Tk"])
    seen = 0
    for b in range(c["B"]):
        mark = np.zeros(c["Tk"] + 1, np.int64)
        live = hi[b] > lo[b]
        np.add.at(mark, lo[b][live], 1)
        np.add.at(mark, hi[b][live], -1)
        seen += int((np.cumsum(mark)[:-1] > 0).sum())
    return int(np.maximum(hi - lo, 0).sum()), seen


def _frequencies(c):
    """Angles per position, in 64 bits: theta^(-2i/rot); `factor` stretches the context by interpolation, and with
    `parts` only where a pair turns seldom over the original 4096 positions (all below 1 turn, none above 4)."""
    i = np.arange(c["rot"] // 2, dtype=np.float64)
    f = 10000.0 ** (-2.0 * i / c["rot"])
    if not c["parts"]:
        return f / c["factor"]
    turns = 4096.0 * f / (2.0 * math.pi)
    keep = np.clip((turns - 1.0) / (4.0 - 1.0), 0.0, 1.0)
    return f * keep + f / c["factor"] * (1.0 - keep)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = TYPES[c["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dt)

    if c["op"] == "rope":
        B, T, d = c["B"], c["T"], c["d"]
        if c["token_major"]:
            q, k = normal(B, T, c["H"], d).transpose(1, 2), normal(B, T, c["Hkv"], d).transpose(1, 2)
        else:
            q, k = normal(B, c["H"], T, d), normal(B, c["Hkv"], T, d)
        first = torch.randint(0, max(1, c["far"] - T + 1), (B, 1), generator=g, device="cuda")
        pos = (first + torch.arange(T, device="cuda")).to(torch.int32)
        s = dict(case=c, q=q, k=k, pos=pos, plan=None)
        if own:
            import exact_tiled_softmax_attn_gb300 as attn
            s["plan"] = attn.rope_plan(c["rot"], interleaved=c["interleaved"], theta=10000.0, factor=c["factor"],
                                       original_length=4096.0 if c["parts"] else 0.0, low_turns=1.0, high_turns=4.0)
        else:
            s["freq"] = torch.from_numpy(_frequencies(c)).cuda()
        return s
    B, H, Hkv, Tq, Tk = c["B"], c["H"], c["Hkv"], c["Tq"], c["Tk"]
    s = dict(case=c, q=normal(B, H, Tq, c["d"]), k=normal(B, Hkv, Tk, c["d"]), v=normal(B, Hkv, Tk, c["dv"]))
    # queries of a trained layer are not as small as normal ones: scores of a few units, some beyond ten
    s["q"] *= 2.0
    if c["op"] == "train":
        s["do"] = normal(B, H, Tq, c["dv"])
    begin, end, pos = _ranges(c)
    for name, x in (("key_begin", begin), ("key_end", end), ("q_pos", pos)):
        s[name] = None if x is None else torch.from_numpy(x.astype(np.int32)).cuda()
    s["slopes"] = torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda") / H).float() if c["bias"] else None
    return s


# ------------------------------------------------------------------ the plain forms

def _turn(x, cos, sin, rot, interleaved):
    x = x.float()
    a, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        u, v = a[..., 0::2], a[..., 1::2]
        y = torch.stack((u * cos - v * sin, v * cos + u * sin), -1).flatten(-2)
    else:
        u, v = a[..., :rot // 2], a[..., rot // 2:]
        y = torch.cat((u * cos - v * sin, v * cos + u * sin), -1)
    return torch.cat((y, rest), -1) if rest.shape[-1] else y


def _rope_plain(s):
    c = s["case"]
    angle = s["pos"].double()[:, None, :, None] * s["freq"]
    cos, sin = angle.cos().float(), angle.sin().float()
    if c["inverse"]:
        sin = -sin
    return [_turn(x, cos, sin, c["rot"], c["interleaved"]).to(x.dtype).contiguous() for x in (s["q"], s["k"])]


def _attention_plain(s):
    c = s["case"]
    G, dt = c["H"] // c["Hkv"], s["q"].dtype
    scale = 1.0 / math.sqrt(c["d"])
    q = s["q"].float()
    k, v = s["k"].float(), s["v"].float()
    B, H, Tq, d = q.shape
    Tk = k.shape[2]
    qg = q.view(B, c["Hkv"], G * Tq, d)                        # the rows of the heads that share a key head
    x = torch.matmul(qg, k.transpose(-1, -2)).mul_(scale).view(B, H, Tq, Tk)
    t = None
    if c["cap"]:
        t = x.div_(c["cap"]).tanh_()
        x = t * c["cap"]
    j = torch.arange(Tk, device=q.device)
    if s["slopes"] is not None:
        x = x - s["slopes"][:, None, None] * (s["q_pos"][:, None, :, None] - j).abs().float()
    if s["key_begin"] is not None:
        x.masked_fill_((j < s["key_begin"][..., None])[:, None], -math.inf)
    if s["key_end"] is not None:
        x.masked_fill_((j >= s["key_end"][..., None])[:, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = x.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    lse = (m + l.log()).squeeze(-1)
    p = p.div_(torch.where(l == 0, torch.ones_like(l), l))
    o = torch.matmul(p.view(B, c["Hkv"], G * Tq, Tk), v).view(B, H, Tq, c["dv"])
    if c["op"] != "train":
        return [o.to(dt), lse]
    do = s["do"].float()
    D = (do * o).sum(-1, keepdim=True)
    dog = do.view(B, c["Hkv"], G * Tq, c["dv"])
    ds = torch.matmul(dog, v.transpose(-1, -2)).view(B, H, Tq, Tk).sub_(D).mul_(p)
    if t is not None:
        ds.mul_(t.square_().neg_().add_(1.0))
    ds = ds.view(B, c["Hkv"], G * Tq, Tk)
    dq = torch.matmul(ds, k).mul_(scale).view(B, H, Tq, d)
    dk = torch.matmul(ds.transpose(-1, -2), qg).mul_(scale)
    dv = torch.matmul(p.view(B, c["Hkv"], G * Tq, Tk).transpose(-1, -2), dog)
    return [o.to(dt), lse, dq.to(dt), dk.to(dt), dv.to(dt)]


def run(state):
    s = state
    c = s["case"]
    if not own:
        return _rope_plain(s) if c["op"] == "rope" else _attention_plain(s)
    import exact_tiled_softmax_attn_gb300 as attn
    if c["op"] == "rope":
        return attn.rope(s["q"], s["k"], s["plan"], pos=s["pos"], inverse=c["inverse"])
    how = dict(softcap=c["cap"], slopes=s["slopes"], q_pos=s["q_pos"], key_begin=s["key_begin"],
               key_end=s["key_end"])
    o, lse = attn.forward_scored(s["q"], s["k"], s["v"], **how)
    if c["op"] != "train":
        return [o, lse]
    return [o, lse, *attn.backward_scored(s["q"], s["k"], s["v"], o, lse, s["do"], **how)]


def work(case):
    c = case
    e = SIZE[c["dtype"]]
    B = c["B"]
    if c["op"] == "rope":
        n = B * c["T"] * (c["H"] + c["Hkv"])
        return {"bytes": 2 * n * c["d"] * e + 4 * B * c["T"], "flops": 3 * n * c["rot"]}
    pairs, seen = _pairs(c)
    H, Hkv, Tq, Tk, d, dv = (c[x] for x in ("H", "Hkv", "Tq", "Tk", "d", "dv"))
    rows = B * H * Tq
    bytes_ = rows * (d + dv) * e + rows * 4 + seen * Hkv * (d + dv) * e + 12 * B * Tq
    flops = 2 * H * pairs * (d + dv)
    if c["op"] == "train":   # dO in, dQ, dK and dV out; the scores again and four products
        bytes_ += rows * (d + dv) * e + B * Hkv * Tk * (d + dv) * e
        flops += 2 * H * pairs * (3 * d + 2 * dv)
    return {"bytes": bytes_, "flops": flops}


# ------------------------------------------------------------------ from the definition, in 64 bits

def _exact_rope(s, c):
    f = torch.as_tensor(_frequencies(c), device="cuda")
    a = torch.einsum("bt,i->bti", s["pos"].to(torch.float64), f)
    z = torch.polar(torch.ones_like(a), -a if c["inverse"] else a)[:, None]      # e^(i angle)
    out = []
    for x in (s["q"], s["k"]):
        x = x.to(torch.float64)
        r, h = c["rot"], c["rot"] // 2
        even = torch.arange(0, r, 2) if c["interleaved"] else torch.arange(h)
        odd = even + (1 if c["interleaved"] else h)
        w = torch.complex(x[..., even], x[..., odd]) * z
        y = x.clone(memory_format=torch.contiguous_format)
        y[..., even], y[..., odd] = w.real, w.imag
        out.append(y)
    return out


def _exact_head(q, k, v, do, c, slope, begin, end, pos):
    """One query head: o, lse and, where do is given, dq and its shares of dk and dv."""
    scale = 1.0 / math.sqrt(c["d"])
    s = scale * (q @ k.mT)
    slope_of_cap = None
    if c["cap"]:
        s = c["cap"] * torch.tanh(s / c["cap"])
        slope_of_cap = 1.0 - (s / c["cap"]) ** 2
    j = torch.arange(k.shape[0], device=q.device)[None, :]
    if slope is not None:
        s = s - slope * (pos[:, None] - j).abs().to(torch.float64)
    off = torch.zeros(s.shape, dtype=torch.bool, device=q.device)
    if begin is not None:
        off |= j < begin[:, None]
    if end is not None:
        off |= j >= end[:, None]
    s[off] = -math.inf
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - torch.nan_to_num(lse, neginf=0.0)[:, None])
    o = p @ v
    if do is None:
        return o, lse
    dp = do @ v.mT
    ds = p * (dp - (do * o).sum(-1)[:, None])
    if slope_of_cap is not None:
        ds = ds * slope_of_cap
    return o, lse, scale * (ds @ k), scale * (ds.mT @ q), p.mT @ do


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "rope":
        return _exact_rope(s, c)
    B, H, G = c["B"], c["H"], c["H"] // c["Hkv"]
    q, k, v = s["q"], s["k"], s["v"]
    f8 = torch.float64
    o = torch.empty(B, H, c["Tq"], c["dv"], dtype=f8, device="cuda")
    lse = torch.empty(B, H, c["Tq"], dtype=f8, device="cuda")
    grads = None
    if c["op"] == "train":
        grads = [torch.zeros(x.shape, dtype=f8, device="cuda") for x in (q, k, v)]
    row = lambda x, b: None if x is None else x[b].long()  # noqa: E731
    for b in range(B):
        for h in range(H):
            slope = None if s["slopes"] is None else s["slopes"][h].to(f8)
            got = _exact_head(q[b, h].to(f8), k[b, h // G].to(f8), v[b, h // G].to(f8),
                              s["do"][b, h].to(f8) if grads else None, c, slope, row(s["key_begin"], b),
                              row(s["key_end"], b), row(s["q_pos"], b))
            o[b, h], lse[b, h] = got[0], got[1]
            if grads:
                grads[0][b, h] = got[2]
                grads[1][b, h // G] += got[3]
                grads[2][b, h // G] += got[4]
    return [o, lse] + (grads or [])
