"""Scored attention and rotary positions in float64: the plain definitions
(test infrastructure).

Scored attention, for query row i of query head h and key j of key head
h // (H / Hkv), with x = scale * q_i . k_j::

    t    = softcap * tanh(x / softcap)        (x itself without a cap)
    S_ij = t - slopes[h] * |pos_i - j|
    S_ij = -inf unless begin_i <= j < end_i and (causal) j <= pos_i
    P = softmax(S),  O = P V,  LSE = log sum exp S     (empty row: O = 0, LSE = -inf)

    dV = P^T dO,  dS = P o (dO V^T - rowsum(dO o O)) o (1 - (t / softcap)^2)
    dQ = scale dS K,  dK = scale dS^T Q       (dK, dV summed over a group's query heads)
"""
from __future__ import annotations

import numpy as np

from .attention import _as64

__all__ = ["scored", "rope_frequencies", "rope"]


def _ints(x, shape, default):
    if x is None:
        return np.broadcast_to(np.asarray(default, np.int64), shape)
    if hasattr(x, "detach"):
        x = x.detach().cpu().numpy()
    return np.asarray(x).astype(np.int64)


def scored(q, k, v, do=None, scale=1.0, causal=False, softcap=0.0, slopes=None, q_pos=None, key_begin=None,
           key_end=None):
    """dict of O, LSE and, with do, dQ, dK, dV."""
    q, k, v = _as64(q), _as64(k), _as64(v)
    B, H, Tq, _ = q.shape
    Hkv, Tk = k.shape[1], k.shape[2]
    G = H // Hkv
    pos = _ints(q_pos, (B, Tq), np.arange(Tq)[None, :])
    lo = np.maximum(_ints(key_begin, (B, Tq), 0), 0)
    hi = np.minimum(_ints(key_end, (B, Tq), Tk), Tk)
    if causal:
        hi = np.minimum(hi, pos + 1)
    j = np.arange(Tk)
    slopes = None if slopes is None else _as64(slopes)
    do = None if do is None else _as64(do)
    out = {"O": np.zeros((B, H, Tq, v.shape[3])), "LSE": np.full((B, H, Tq), -np.inf)}
    if do is not None:
        out.update(dQ=np.zeros_like(q), dK=np.zeros_like(k), dV=np.zeros_like(v))
    for b in range(B):
        seen = (j >= lo[b][:, None]) & (j < hi[b][:, None])
        live = seen.any(axis=1)
        for h in range(H):
            kh, vh = np.where(seen.any(axis=0)[:, None], k[b, h // G], 0), np.where(seen.any(axis=0)[:, None], v[b, h // G], 0)
            s = scale * (q[b, h] @ kh.T)
            slope = 1.0
            if softcap:
                t = np.tanh(s / softcap)
                s, slope = softcap * t, 1.0 - t * t
            if slopes is not None:
                s = s - slopes[h] * np.abs(pos[b][:, None] - j)
            s = np.where(seen, s, -np.inf)
            m = np.where(live, s.max(axis=1, initial=-np.inf), 0.0)
            p = np.exp(s - m[:, None])
            l = np.where(live, p.sum(axis=1), 1.0)
            p /= l[:, None]
            o = p @ vh
            out["O"][b, h] = o
            out["LSE"][b, h] = np.where(live, m + np.log(l), -np.inf)
            if do is not None:
                g = do[b, h]
                ds = p * (g @ vh.T - (g * o).sum(axis=1)[:, None]) * slope
                out["dQ"][b, h] = scale * (ds @ kh)
                out["dK"][b, h // G] += scale * (ds.T @ q[b, h])
                out["dV"][b, h // G] += p.T @ g
    return out


def rope_frequencies(rot, theta=10000.0, factor=1.0, original_length=0.0, low_turns=1.0, high_turns=4.0):
    f = theta ** (-2.0 * np.arange(rot // 2) / rot)
    keep = np.zeros_like(f)
    if original_length > 0:
        keep = np.clip((original_length * f / (2 * np.pi) - low_turns) / (high_turns - low_turns), 0.0, 1.0)
    return f * keep + f / factor * (1.0 - keep)


def rope(x, pos, freq, interleaved=False, inverse=False, mscale=1.0):
    """x [B, H, T, d] turned by pos [B, T] * freq [rot / 2]."""
    x = _as64(x)
    y = x.copy()
    n = len(freq)
    a = np.asarray(pos, np.float64)[:, None, :, None] * freq
    c, s = mscale * np.cos(a), mscale * np.sin(a) * (-1.0 if inverse else 1.0)
    iu = np.arange(n) * 2 if interleaved else np.arange(n)
    iv = iu + (1 if interleaved else n)
    u, v = x[..., iu], x[..., iv]
    y[..., iu], y[..., iv] = u * c - v * s, v * c + u * s
    return y
