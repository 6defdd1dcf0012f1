"""Paged INT4 KV cache, norm and rotation of q and k, and attention over the cache, in
float64 numpy: the CPU reference of the attention side.

Plain readings of the formulas: a token's K and V rows are quantized by the KV rule of
kv.py, stored at (page, row), and attention is the softmax of scaled dot products over
the dequantized values. `tile_bytes` follows the written byte layout one code at a time.
"""

from __future__ import annotations

import numpy as np

from .kv import dequant_kv_int4, quantize_kv_int4


def rope_angles(positions, rot: int, theta: float = 10000.0) -> np.ndarray:
    """position * theta^(-2 i / rot), float64 [len(positions), rot / 2]."""
    i = np.arange(rot // 2, dtype=np.float64)
    return np.asarray(positions, dtype=np.float64)[:, None] * np.power(float(theta), -2.0 * i / rot)


def norm_rope(x, weight=None, eps: float = 1e-6, cos=None, sin=None, interleaved: bool = False) -> np.ndarray:
    """float64 [tokens, heads, d]: RMS norm of each head (no weight: none), then the pairs
    (i, i + r) or (2i, 2i + 1), i < r = cos.shape[1], turned by cos + j sin."""
    y = np.asarray(x).astype(np.float64)
    if weight is not None:
        y = y / np.sqrt(np.mean(y * y, axis=-1, keepdims=True) + eps) * np.asarray(weight).astype(np.float64)
    if cos is None:
        return y
    out = y.copy()
    half = cos.shape[1]
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = (np.asarray(t[:, i], dtype=np.float64)[:, None] for t in (cos, sin))
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., b] * c + y[..., a] * s
    return out


def store(x, group: int):
    """Codes and scales of token rows [tokens, heads, d] float16, and the values they stand
    for (float64)."""
    q, s = quantize_kv_int4(np.asarray(x)[None], group)
    return q[0], s[0], dequant_kv_int4(q, s, group)[0]


def tile_bytes(codes, is_v: bool) -> np.ndarray:
    """The bytes of one tile: codes int [16 tokens, d] -> uint8 [8 d]."""
    d = codes.shape[1]
    n_dw = min(d // 32, 4)
    words = [0] * (2 * d)
    for t in range(16):
        for ch in range(d):
            m = ch // 32
            nib = int(codes[t, ch]) + 8
            if is_v:
                n, r = ch % 32 // 16, ch % 16
                lane = r + 16 * (t // 4)
                bit = 8 * (0, 2, 1, 3)[t % 4] + 4 * n
            else:
                c, e = ch % 32 // 8, ch % 8
                lane = t + 16 * c
                bit = 4 * (e // 2 if e % 2 == 0 else 4 + (e - 1) // 2)
            words[(m // n_dw * 64 + lane) * n_dw + m % n_dw] |= nib << bit
    return np.array(words, dtype="<u4").view(np.uint8)


def attention(q, k, v, lens, offsets, scale: float, window: int = 0) -> np.ndarray:
    """float64 [tokens, q_heads, d]. Sequence n's rows are offsets[n] .. offsets[n + 1] - 1, the
    last of its lens[n] tokens; k[n], v[n]: float64 [lens[n], kv_heads, d]. A row that sees
    nothing is zero; rows of no sequence are NaN."""
    q = np.asarray(q).astype(np.float64)
    out = np.full(q.shape, np.nan)
    for n, length in enumerate(lens):
        first, last = offsets[n], offsets[n + 1]
        share = q.shape[1] // k[n].shape[1]
        for i in range(first, last):
            pos = length - (last - first) + (i - first)
            lo = max(0, pos - window + 1) if window else 0
            for h in range(q.shape[1]):
                kh, vh = k[n][lo:pos + 1, h // share], v[n][lo:pos + 1, h // share]
                if pos < lo or pos < 0:
                    out[i, h] = 0.0
                    continue
                z = kh @ q[i, h] * scale
                p = np.exp(z - z.max())
                out[i, h] = (p / p.sum()) @ vh
    return out
