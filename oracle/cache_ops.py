"""Float64 oracle of the calls in include/gqa_cache.h (test infrastructure, as the rest of this package).

Plain numpy in double, one loop per sequence and KV head, from the formulas in
the header; bfloat16 arrays are uint16 bit patterns, as everywhere here. The
eviction and the 4-bit format are exact and are written as searches (a sort of
tuples, the nearest of eight candidates), not as the bit tricks of a kernel.
"""
from __future__ import annotations

import numpy as np

from . import widen

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def rope_table(max_pos: int, rotary_dim: int, theta: float) -> np.ndarray:
    i = np.arange(rotary_dim // 2, dtype=np.float64)
    a = np.arange(max_pos, dtype=np.float64)[:, None] * theta ** (-2.0 * i / max(rotary_dim, 1))[None, :]
    return np.concatenate([np.cos(a), np.sin(a)], axis=1)


def norm_heads(x, weight, eps: float) -> np.ndarray:
    """x [..., d] -> x / sqrt(mean x^2 + eps) * weight (weight None: x)."""
    x = widen(x)
    if weight is None:
        return x
    return x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * widen(weight)


def rotate(y, table, positions, interleaved: bool) -> np.ndarray:
    """y [B, T, heads, d] float64, table [max_pos, rotary_dim] (None: no rotation), positions [B, T] inside it."""
    if table is None or table.shape[1] == 0:
        return y
    r = table.shape[1]
    z = y.copy()
    row = np.asarray(table, np.float64)[np.asarray(positions)]
    cos, sin = row[:, :, None, :r // 2], row[:, :, None, r // 2:]
    lo = slice(0, r, 2) if interleaved else slice(0, r // 2)
    hi = slice(1, r, 2) if interleaved else slice(r // 2, r)
    a, b = y[..., lo], y[..., hi]
    z[..., lo] = a * cos - b * sin
    z[..., hi] = b * cos + a * sin
    return z


def softmax_weights(q, keys, scale: float) -> np.ndarray:
    """q [h, d], keys [n, d] float64 -> softmax over the keys [h, n]."""
    x = scale * (q @ keys.T)
    e = np.exp(x - x.max(axis=1, keepdims=True))
    return e / e.sum(axis=1, keepdims=True)


def decode_scores(q, k_cache, v_cache, seqlens, scale: float):
    """(out [B, H, d], added [B, K, S_max], spread [B, H, d]): the outputs, what each row's score gains, and
    sum_t p |v|, the size that the rounding of p acts on."""
    q, k, v = widen(q), widen(k_cache), widen(v_cache)
    B, H, d = q.shape
    K, S = k.shape[1:3]
    G = H // K
    out, spread, added = np.zeros((B, H, d)), np.zeros((B, H, d)), np.zeros((B, K, S))
    for b in range(B):
        n = int(seqlens[b])
        if n == 0:
            continue
        for g in range(K):
            h = slice(g * G, (g + 1) * G)
            p = softmax_weights(q[b, h], k[b, g, :n], scale)
            out[b, h] = p @ v[b, g, :n]
            spread[b, h] = p @ np.abs(v[b, g, :n])
            added[b, g, :n] = p.sum(axis=0)
    return out, added, spread


def prompt_scores(q, k_cache, seqlens, scale: float) -> np.ndarray:
    """q [B, T, H, d] -> what each row's score gains [B, K, S_max]."""
    q, k = widen(q), widen(k_cache)
    B, T, H, d = q.shape
    K, S = k.shape[1:3]
    G = H // K
    added = np.zeros((B, K, S))
    for b in range(B):
        for i in range(T):
            n = int(seqlens[b]) - T + i + 1  # keys that query i sees
            if n <= 0:
                continue
            for g in range(K):
                added[b, g, :n] += softmax_weights(q[b, i, g * G:(g + 1) * G], k[b, g, :n], scale).sum(axis=0)
    return added


def evict(k_cache, v_cache, scores, row_pos, seqlens, keep: int, sinks: int, recent_from):
    """Copies of (k_cache, v_cache, scores, row_pos, seqlens) after the eviction; row_pos may be None."""
    k, v, s = k_cache.copy(), v_cache.copy(), scores.copy()
    pos = None if row_pos is None else row_pos.copy()
    lens = np.array(seqlens, np.int32)
    B, K, S = scores.shape
    for b in range(B):
        n = int(lens[b])
        if n <= keep or n > S:
            continue
        for g in range(K):
            where = np.arange(n) if pos is None else row_pos[b, g, :n].astype(np.int64)
            held = where < sinks
            if recent_from is not None:
                held |= where >= int(recent_from[b])

            def rank(t):
                w = float(scores[b, g, t])
                return (0, 0.0, t) if held[t] else (1, -w, t) if w == w else (2, 0.0, t)

            stay = sorted(range(n), key=rank)[:keep]
            movers = sorted(t for t in stay if t >= keep)
            holes = sorted(set(range(keep)) - set(stay))
            assert len(movers) == len(holes)
            for a in (k, v):
                a[b, g, holes] = a[b, g, movers]
            s[b, g, holes] = s[b, g, movers]
            s[b, g, keep:n] = 0.0
            if pos is not None:
                pos[b, g, holes] = pos[b, g, movers]
                pos[b, g, keep:n] = -1
        lens[b] = keep
    return k, v, s, pos, lens


def mxfp4_quantize(x):
    """x [..., d] (d a multiple of 32) -> codes [..., d / 2] uint8, scales [..., d / 32] uint8."""
    x = widen(x)
    blocks = x.reshape(*x.shape[:-1], -1, 32)
    top = np.max(np.abs(blocks), axis=-1)
    bad = ~np.isfinite(top)
    m, e = np.frexp(np.where(bad, 0.0, top))  # top = m 2^e, 0.5 <= m < 1
    E = np.clip(np.where(top == 0, -127, e - 1 - 2), -127, 127) + 127
    step = np.ldexp(1.0, E - 127)[..., None]
    with np.errstate(invalid="ignore"):
        a = np.abs(blocks) / step
    code = np.zeros(blocks.shape, np.int64)
    far = np.full(blocks.shape, np.inf)
    for c in (0, 2, 4, 6, 1, 3, 5, 7):  # the even codes first: they win ties
        d = np.abs(np.where(np.isfinite(a), a, 0.0) - E2M1[c])
        code = np.where(d < far, c, code)
        far = np.minimum(far, d)
    code += 8 * np.signbit(blocks)
    code = np.where(bad[..., None], 0, code).reshape(x.shape)
    E = np.where(bad, 255, E)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8), E.astype(np.uint8)


def mxfp4_values(codes, scales) -> np.ndarray:
    """What a 4-bit cache holds, float64 (NaN for scale 255)."""
    both = np.stack([codes & 15, codes >> 4], axis=-1).reshape(*codes.shape[:-1], -1).astype(np.int64)
    value = np.array(E2M1 + tuple(-v for v in E2M1))[both]
    step = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return value * np.repeat(step, 32, axis=-1)
