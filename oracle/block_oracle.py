"""Plain fp64 CPU oracle of a decoder block's attention half: the norms with the residual, the
rotary split, attention over packed prompts, the 4-bit cache and attention over it.

TEST INFRASTRUCTURE ONLY, like gptq_oracle (whose group parameters and codes the cache shares:
gptq_quantize_layer's asymmetric grid).  numpy only; nothing of the library is used.
"""
from __future__ import annotations

from typing import Optional

import numpy as np

from .gptq_oracle import group_params, quantize_codes


def norm(v, w, b, eps: float, center: bool):
    """v / sqrt(mean(v^2) + eps) . w + b per row; of v - mean(v) with center."""
    v = np.asarray(v, np.float64)
    if center:
        v = v - v.mean(-1, keepdims=True)
    y = v / np.sqrt((v * v).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    return y if b is None else y + np.asarray(b, np.float64)


def add(x, y, gate, alpha: float, post_w=None, post_b=None, eps: float = 1e-6, center: bool = False):
    """x + alpha . gate . N(y; post) before its rounding."""
    y = np.asarray(y, np.float64)
    if post_w is not None:
        y = norm(y, post_w, post_b, eps, center)
    if gate is not None:
        y = y * np.asarray(gate, np.float64)
    return np.asarray(x, np.float64) + alpha * y


def rope_qkv(x, cos, sin, heads_q: int, heads_kv: int, d: int, positions, bias=None, interleaved: bool = False):
    """(q, k, v) [tokens, heads, d] of x [tokens, (heads_q + 2 heads_kv) d]."""
    x = np.array(x, np.float64)
    if bias is not None:
        x = x + np.asarray(bias, np.float64)
    x = x.reshape(x.shape[0], heads_q + 2 * heads_kv, d)
    if cos is not None:
        half = cos.shape[1]
        for t, p in enumerate(positions):
            for i in range(half):
                i0, i1 = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
                c, s = float(cos[p, i]), float(sin[p, i])
                a, b = x[t, :heads_q + heads_kv, i0].copy(), x[t, :heads_q + heads_kv, i1].copy()
                x[t, :heads_q + heads_kv, i0] = a * c - b * s
                x[t, :heads_q + heads_kv, i1] = a * s + b * c
    return x[:, :heads_q], x[:, heads_q:heads_q + heads_kv], x[:, heads_q + heads_kv:]


def attend(q, k, v, scale: float, seen):
    """(o, weights' sum of p |v|) of q [n, d] against k, v [m, d]; seen[i] = how many of the first keys
    query i sees.  Keys that are not seen take no part; a query that sees none gives 0."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    o, mag = np.zeros((q.shape[0], v.shape[1])), np.zeros((q.shape[0], v.shape[1]))
    for i in range(q.shape[0]):
        n = int(max(0, min(seen[i], k.shape[0])))
        if n == 0:
            continue
        s = scale * (k[:n] @ q[i])
        p = np.exp(s - s.max())
        p /= p.sum()
        o[i] = p @ v[:n]
        mag[i] = p @ np.abs(v[:n])
    return o, mag


def attention(q, k, v, cu_q, cu_k, scale: float, causal: bool):
    """(o, mag) [total_q, heads_q, d]; rows of no sequence stay NaN in o."""
    hq, hk = q.shape[1], k.shape[1]
    o = np.full(q.shape, np.nan)
    mag = np.zeros(q.shape)
    for b in range(len(cu_q) - 1):
        q0, q1, k0, k1 = cu_q[b], cu_q[b + 1], cu_k[b], cu_k[b + 1]
        lq, lk = q1 - q0, k1 - k0
        seen = [lk if not causal else i + 1 + lk - lq for i in range(lq)]
        for h in range(hq):
            g = h // (hq // hk)
            o[q0:q1, h], mag[q0:q1, h] = attend(q[q0:q1, h], k[k0:k1, g], v[k0:k1, g], scale, seen)
    return o, mag


def kv4_quantize(x, group: int):
    """x [..., d] -> codes [..., d], scales and zero points [..., d / group] (fp32 values)."""
    x = np.asarray(x, np.float32)
    g = x.reshape(-1, group)
    s, z = group_params(g, 4, False)
    c = np.stack([quantize_codes(g[:, i], s, z, 4, False) for i in range(group)], 1)
    par = x.shape[:-1] + (x.shape[-1] // group,)
    return c.reshape(x.shape), s.reshape(par), z.reshape(par)


def kv4_values(codes, scales, zeros):
    """s (c - z) in fp64."""
    c = np.asarray(codes, np.float64)
    g = c.reshape(scales.shape + (c.shape[-1] // scales.shape[-1],))
    return (np.asarray(scales, np.float64)[..., None] * (g - np.asarray(zeros, np.float64)[..., None])).reshape(c.shape)


def kv4_words(codes):
    """codes [..., d] -> uint32 words [..., d / 8]: code i of a word in bits 4 i .. 4 i + 3."""
    c = np.asarray(codes, np.uint64)
    c = c.reshape(c.shape[:-1] + (c.shape[-1] // 8, 8))
    return (c << (4 * np.arange(8, dtype=np.uint64))).sum(-1).astype(np.uint32)
