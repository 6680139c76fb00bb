"""The INT4 cache row by its definition, in numpy, and problems of the decode over such pages."""
from __future__ import annotations

import math

import numpy as np

import mla_workloads as mw

SCALE = 1.0 / math.sqrt(192.0)


def wide(bits):
    """float32 of bf16 bits."""
    return (np.asarray(bits).astype(np.uint32) << 16).view(np.float32)


def quantize_rows(lat, rope_bits):
    """Latent values (bf16 numbers, [n, 512]) and RoPE bits [n, 64] -> rows [n, 416] by the rule of mla_quantize_kv_int4."""
    g = np.asarray(lat, np.float32).reshape(-1, 16, 32)
    with np.errstate(all="ignore"):
        top = np.abs(g).max(-1)
        bad = ~np.isfinite(g).all(-1)
        s = ((top / np.float32(7)).astype(np.float32).view(np.uint32) + np.uint32(0xFFFFF) & np.uint32(0xFFF00000)).view(np.float32)
        s = np.maximum(s, np.float32(2.0 ** -126))
        bad |= ~(s <= np.float32(2.0 ** 119))
        s = np.where((top == 0) | bad, np.float32(1), s)
        n = np.rint(g / s[..., None]) + 8
    n = np.where(bad[..., None], 8, n).astype(np.uint32).reshape(-1, 64, 8)
    word = np.zeros(n.shape[:2], np.uint32)
    for k in range(8):
        word |= n[..., k] << np.uint32(4 * (k // 2) + 16 * (k % 2))
    bits = np.where(bad, np.uint16(0x7FC0), (s.view(np.uint32) >> 16).astype(np.uint16)).astype(np.uint16)
    rope = np.ascontiguousarray(rope_bits, np.uint16).reshape(-1, 64)
    return np.concatenate([word.view(np.uint8).reshape(-1, 256), bits.view(np.uint8).reshape(-1, 32), rope.view(np.uint8).reshape(-1, 128)], 1)


def dequantize_rows(raw):
    """Rows [n, 416] -> float64 [n, 576]."""
    raw = np.ascontiguousarray(raw).reshape(-1, 416)
    word = np.ascontiguousarray(raw[:, :256]).view(np.uint32)
    s = wide(np.ascontiguousarray(raw[:, 256:288]).view(np.uint16)).astype(np.float64)
    lat = np.empty((len(raw), 64, 8))
    for k in range(8):
        lat[..., k] = (word >> np.uint32(4 * (k // 2) + 16 * (k % 2)) & np.uint32(15)).astype(np.float64) - 8
    with np.errstate(invalid="ignore"):
        lat = lat.reshape(-1, 16, 32) * s[..., None]
    return np.concatenate([lat.reshape(-1, 512), wide(np.ascontiguousarray(raw[:, 288:]).view(np.uint16)).astype(np.float64)], 1)


def random_rows(rng, n, spread=0.0):
    """Rows of N(0, 1) latents and RoPE keys, each token's latents times exp(spread * N(0, 1))."""
    x = rng.standard_normal((n, 576), dtype=np.float32)
    x[:, :512] *= np.exp(spread * rng.standard_normal((n, 1), dtype=np.float32))
    bits = mw.to_bf16_bits(x)
    return quantize_rows(wide(bits[:, :512]), bits[:, 512:])


def place(rng, L, extra=3):
    """(pages in all, block table): a random page for each that the lengths need, -1 elsewhere."""
    need = -(-np.maximum(L, 0) // 64)
    P = int(need.sum()) + extra
    perm, bt, o = rng.permutation(P).astype(np.int32), np.full((len(L), max(1, int(need.max()))), -1, np.int32), 0
    for b, k in enumerate(need):
        bt[b, :k] = perm[o:o + k]
        o += k
    return P, bt


def reference(q, qr, rows, seen, scale=SCALE):
    """One token over `seen` of the rows: (out [H, 512], lse [H], bounds of |out error| and |lse error|), in float64.

    The bounds, with w the softmax weights and A = sum_j w_j |c_j|: a score is a float32 sum of 576 exact products, each partial
    sum off by at most 2^-23 of its size, so |score error| <= d = scale * 576 * 2^-23 * max_j sum_i |q_i k_ji|.  lse moves by at
    most d, 2^-20 (the last logarithm and products, exponentials of 2 ulp) and 2^-23 of its size.  A weight is off by at most
    2 d and by 2^-8 (P in bf16), the output is rounded to bf16, 2^-8 of its size at most (float32 outputs need less):
    |out error| <= 2^-8 |out| + (2^-8 + 2 d + 2^-14) A, 2^-14 covering float32 accumulation, rescaling and division.
    That holds while nothing underflows.  The exponential gives 0 below 2^-126, of a weight relative to a maximum that some key
    has (so that the sum is at least 1): a weight is then off by at most 2^-126, and the output by 2^-126 sum_j |c_j| more, which is
    above half a step of bf16's least numbers, too."""
    H = len(q)
    if seen <= 0:
        return np.zeros((H, 512)), np.full(H, -np.inf), np.zeros((H, 512)), np.zeros(H)
    c, key, x = rows[:seen, :512], rows[:seen], np.concatenate([q, qr], 1)
    s = scale * (x @ key.T)
    m = s.max(1, keepdims=True)
    e = np.exp(s - m)
    z = e.sum(1, keepdims=True)
    w = e / z
    out, lse = w @ c, (m + np.log(z))[:, 0]
    d = scale * 576 * 2.0 ** -23 * (np.abs(x) @ np.abs(key).T).max(1)
    return out, lse, 2.0 ** -8 * np.abs(out) + (2.0 ** -8 + 2 * d[:, None] + 2.0 ** -14) * (w @ np.abs(c)) + 2.0 ** -126 * np.abs(c).sum(0), d + 2.0 ** -20 + 2.0 ** -23 * np.abs(lse)
