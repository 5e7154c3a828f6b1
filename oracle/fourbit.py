"""fp64 CPU oracle of the 4-bit cache, of the normalised append with positions
of several axes, and of attention over cached rows given as values.

A 4-bit row is (codes 0..15, scale, minimum), value minimum + scale * code.
The scale is found here by search over the bf16 numbers, the codes by division
in float64: differences of two bf16 values and products of a bf16 value and a
half-integer below 16 differ, where they differ at all, by more than 2^-45 of
themselves, so no quotient is rounded across a half.
"""

from __future__ import annotations

import numpy as np

from .decode import F64, rope_inv_freq, round_bf16


def bf16_bits(x) -> np.ndarray:
    """uint16 bit patterns of bf16 values."""
    return (np.asarray(x, np.float32).view(np.uint32) >> 16).astype(np.uint16)


def bf16_from_bits(b) -> np.ndarray:
    return (np.asarray(b).astype(np.uint32) << 16).view(np.float32).astype(F64)


def quantize_u4(x):
    """Rows (last axis) of bf16 values -> (codes uint8 [..., d], scale [...], minimum [...])."""
    bad = ~np.isfinite(np.asarray(x, F64)).all(-1)
    x = np.clip(np.nan_to_num(np.asarray(x, F64), nan=0.0), -2.0 ** 126, 2.0 ** 126)
    lo, hi = x.min(-1), x.max(-1)
    lo = lo + 0.0  # no -0
    span = hi - lo + 0.0
    bits = bf16_bits(round_bf16(span / 15)).astype(np.int64)
    for _ in range(2):  # to the smallest bf16 that reaches the maximum
        bits = np.where(bf16_from_bits(bits) * 15 < span, bits + 1, bits)
        below = np.maximum(bits - 1, 0)
        bits = np.where((bits > 0) & (bf16_from_bits(below) * 15 >= span), below, bits)
    scale = bf16_from_bits(bits)
    with np.errstate(all="ignore"):
        q = (x - lo[..., None]) / np.where(scale == 0, 1.0, scale)[..., None]
        codes = np.where(bad[..., None], 0, np.clip(np.rint(q), 0, 15)).astype(np.uint8)
    return codes, np.where(bad, np.nan, scale), np.where(bad, 0.0, lo)


def pack_u4(codes) -> np.ndarray:
    """[..., d] codes -> [..., d / 2] bytes, the even element in the low half."""
    c = np.asarray(codes, np.uint8)
    return c[..., 0::2] | c[..., 1::2] << 4


def unpack_u4(packed) -> np.ndarray:
    p = np.asarray(packed, np.uint8)
    return np.stack([p & 15, p >> 4], -1).reshape(*p.shape[:-1], -1)


def dequantize_u4(codes, scale, low) -> np.ndarray:
    return np.asarray(low, F64)[..., None] + np.asarray(scale, F64)[..., None] * np.asarray(codes, F64)


def norm_rope(x, weight, eps: float, positions, sections, base: float) -> np.ndarray:
    """x [..., d] normalised (weight None: not) and turned: positions[a] the position of axis a, sections[a] its pairs."""
    x = np.asarray(x, F64)
    if weight is not None:
        x = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * np.asarray(weight, F64)
    at = np.concatenate([np.full(w, float(p)) for p, w in zip(positions, sections)])
    z = (x[..., 0::2] + 1j * x[..., 1::2]) * np.exp(1j * at * rope_inv_freq(x.shape[-1], base))
    return np.stack([z.real, z.imag], -1).reshape(x.shape)


def attention_values(q, K, V, first: int, scale: float, window: int = 0):
    """q [n, Hq, d] whose token i is at position first + i and sees the keys [0, first + i] (the last `window`); K, V
    [Hkv, L, d] values. Returns (out [n, Hq, d], lse [n, Hq])."""
    q, K, V = (np.asarray(t, F64) for t in (q, K, V))
    n, hq, d = q.shape
    g = hq // K.shape[0]
    out, lse = np.empty((n, hq, d)), np.empty((n, hq))
    for i in range(n):
        end = first + i + 1
        begin = max(0, end - window) if window else 0
        for h in range(hq):
            s = scale * (K[h // g, begin:end] @ q[i, h])
            top = s.max()
            p = np.exp(s - top)
            out[i, h] = p @ V[h // g, begin:end] / p.sum()
            lse[i, h] = top + np.log(p.sum())
    return out, lse
