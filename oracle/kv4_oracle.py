"""fp64 oracle of the query/key preparation and of the 4-bit K/V cache (test infrastructure).

Plain numpy statements of the contracts in include/std_b200.h: RMS norm and rotation of query
and key heads, the 4-bit row format (fp32 where the format's definition says so), its byte
layout, and causal decode attention over such a cache.
"""
from __future__ import annotations

from typing import Optional, Sequence, Tuple

import numpy as np

GROUP = 64


def bf16_round(x: np.ndarray) -> np.ndarray:
    """float32 -> nearest bfloat16 (ties to even), as float32; infinities and NaN pass."""
    x = np.ascontiguousarray(x, dtype=np.float32)
    u = x.view(np.uint32).astype(np.uint64)
    r = ((u + 0x7fff + ((u >> 16) & 1)) & 0xffff0000).astype(np.uint32).view(np.float32).reshape(x.shape)
    return np.where(np.isnan(x), np.float32(np.nan), r)


def norm_rope(x: np.ndarray, weight: Optional[np.ndarray], eps: float, pos: np.ndarray, inv_freq: np.ndarray,
              sections: Sequence[int], interleaved: bool) -> np.ndarray:
    """x [n][H][d], pos [axes][n] -> the rotated (and, with a weight [d], normalised) heads."""
    x = np.array(x, dtype=np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    half = len(inv_freq)
    axis = np.repeat(np.arange(len(sections)), sections)
    assert len(axis) == half
    for i in range(half):
        t = pos[axis[i]].astype(np.float64)[:, None] * inv_freq[i]
        u, v = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        a, b = x[..., u].copy(), x[..., v].copy()
        x[..., u] = a * np.cos(t) - b * np.sin(t)
        x[..., v] = b * np.cos(t) + a * np.sin(t)
    return x


def kv4_quantize(x: np.ndarray) -> Tuple[np.ndarray, np.ndarray, np.ndarray]:
    """[..., d] -> codes uint8 [..., d], scale and minimum float32 [..., d / 64]."""
    g = np.asarray(x, dtype=np.float32).reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    with np.errstate(all="ignore"):
        m = bf16_round(g.min(-1))
        span = g.max(-1) - m
        s = bf16_round(np.maximum(span, 0) / np.float32(15))  # (fp32 input: m may round above max x)
        diff = (g - m[..., None]).astype(np.float64)
        c = np.clip(np.round(diff / s[..., None].astype(np.float64)), 0, 15)
    bad = ~np.isfinite(span)
    m = np.where(bad, np.float32(np.nan), m)
    s = np.where(bad, np.float32(0), s)
    c = np.where((s > 0)[..., None], c, 0)
    return c.astype(np.uint8).reshape(x.shape), s, m


def kv4_values(codes: np.ndarray, s: np.ndarray, m: np.ndarray) -> np.ndarray:
    g = codes.reshape(*codes.shape[:-1], codes.shape[-1] // GROUP, GROUP).astype(np.float64)
    return (m[..., None].astype(np.float64) + g * s[..., None].astype(np.float64)).reshape(codes.shape)


def kv4_byte(d: int, channel: int) -> Tuple[int, int]:
    """(byte of a row, shift) of a channel's code."""
    group, c = divmod(channel, GROUP)
    word = (c // 8) * (d // GROUP) + group
    bit = 32 * word + 4 * (c % 8)
    return bit // 8, bit % 8


def kv4_pack(codes: np.ndarray) -> np.ndarray:
    d = codes.shape[-1]
    out = np.zeros(codes.shape[:-1] + (d // 2,), np.uint8)
    for c in range(d):
        byte, shift = kv4_byte(d, c)
        out[..., byte] |= (codes[..., c] << shift).astype(np.uint8)
    return out


def kv4_unpack(packed: np.ndarray) -> np.ndarray:
    d = 2 * packed.shape[-1]
    out = np.zeros(packed.shape[:-1] + (d,), np.uint8)
    for c in range(d):
        byte, shift = kv4_byte(d, c)
        out[..., c] = (packed[..., byte] >> shift) & 15
    return out


def causal_decode_attn(q: np.ndarray, k: np.ndarray, v: np.ndarray, first: np.ndarray) -> np.ndarray:
    """q [L][B][Hq][rows][d], k and v [L][B][Hkv][cap][d] -> o: row i of sequence b attends keys
    j < first[b] + i; a row without keys gives zeros."""
    L, B, Hq, rows, d = q.shape
    G = Hq // k.shape[2]
    o = np.zeros(q.shape, np.float64)
    for l in range(L):
        for b in range(B):
            for h in range(Hq):
                for i in range(rows):
                    n = int(first[b]) + i
                    if n <= 0:
                        continue
                    x = k[l, b, h // G, :n].astype(np.float64) @ q[l, b, h, i].astype(np.float64) / np.sqrt(d)
                    p = np.exp(x - x.max())
                    o[l, b, h, i] = p @ v[l, b, h // G, :n] / p.sum()
    return o
