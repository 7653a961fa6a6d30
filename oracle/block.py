"""The operators around the layer: residual RMS norm and its gradient, rows of
8-bit integers, and the product of such rows (oracle side).

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

Definitions (``include/twell.h``), for storage tensors x, residual, weight:

* h = round(x + residual): one fp32 addition, then the storage rounding.
* y = h / sqrt(mean(h^2) + eps) * weight, here in float64 and unrounded.
* 8 bits of z = h * weight (an fp32 product): m = max(max|z|, 2^-100),
  q = rint(z * (127 / m)), one fp32 rounding per operation, ties to even; the
  values stand for q * scale with scale = m / 127 / sqrt(mean(h^2) + eps), in
  float64.  A row with an infinite or NaN z: q = 0, scale NaN.
* gradient: dx = dh + r g - r^3 h mean(g h) with g = dy * weight and r the
  norm's factor; dweight = sum over rows of dy h r; float64, unrounded.
* product: integer sums, then scales and bias in float64.
"""

from __future__ import annotations

import numpy as np

from .numerics import decode, round_to_storage

TINY = np.float32(2.0 ** -100)


def residual_sum(x: np.ndarray, residual, dtype: str) -> np.ndarray:
    """round(x + residual) as a storage tensor (x itself without a residual)."""
    if residual is None:
        return x
    with np.errstate(all="ignore"):
        s = decode(x, dtype).astype(np.float32) + decode(residual, dtype).astype(np.float32)
    return s if dtype == "f32" else round_to_storage(s.astype(np.float64), dtype)


def norm_factor(h: np.ndarray, eps: float, dtype: str) -> np.ndarray:
    """r_t = 1 / sqrt(mean_j h_tj^2 + eps), float64 [T]."""
    H = decode(h, dtype)
    with np.errstate(all="ignore"):
        return 1.0 / np.sqrt(np.mean(H * H, axis=1) + eps)


def rmsnorm(h: np.ndarray, weight: np.ndarray, eps: float, dtype: str) -> np.ndarray:
    """h * r * weight in float64 (unrounded)."""
    with np.errstate(all="ignore"):
        return decode(h, dtype) * norm_factor(h, eps, dtype)[:, None] * decode(weight, dtype)


def quantize(z: np.ndarray, r: np.ndarray):
    """(q int8, scale float64) of fp32 rows z whose values are z * r[:, None]."""
    z = np.asarray(z, np.float32)
    with np.errstate(all="ignore"):
        top = np.max(np.abs(z), axis=1)
        bad = ~np.isfinite(z).all(axis=1)
        m = np.maximum(np.where(bad, np.float32(1), top), TINY).astype(np.float32)
        inv = (np.float32(127) / m).astype(np.float32)
        v = np.rint((np.where(bad[:, None], np.float32(0), z) * inv[:, None]).astype(np.float32))
    scale = np.where(bad, np.nan, np.asarray(r, np.float64) * m.astype(np.float64) / 127.0)
    return v.astype(np.int8), scale


def rmsnorm_quantized(h: np.ndarray, weight: np.ndarray, eps: float, dtype: str):
    """(q int8, scale float64) of the normed rows."""
    with np.errstate(all="ignore"):
        z = decode(h, dtype).astype(np.float32) * decode(weight, dtype).astype(np.float32)
    return quantize(z, norm_factor(h, eps, dtype))


def quantize_rows(x: np.ndarray, dtype: str):
    """(q int8, scale float64) of x's rows."""
    return quantize(decode(x, dtype).astype(np.float32), np.ones(x.shape[0]))


def rmsnorm_backward(dy: np.ndarray, h: np.ndarray, weight: np.ndarray, eps: float, dtype: str, dh=None):
    """(dx, dweight) in float64, unrounded."""
    H, DY, w = decode(h, dtype), decode(dy, dtype), decode(weight, dtype)
    r = norm_factor(h, eps, dtype)[:, None]
    g = DY * w
    dx = r * g - r ** 3 * H * np.mean(g * H, axis=1, keepdims=True)
    if dh is not None:
        dx = dx + decode(dh, dtype)
    return dx, np.sum(DY * H * r, axis=0)


def int8_matmul(a: np.ndarray, a_scale: np.ndarray, b: np.ndarray, b_scale: np.ndarray, row_bias=None):
    """(sum_k a b) * a_scale * b_scale + row_bias in float64 (the sums exact)."""
    # every partial sum of products of 8-bit integers is a whole number far below 2^53
    s = a.astype(np.float64) @ b.astype(np.float64).T
    y = s * np.asarray(a_scale, np.float64)[:, None] * np.asarray(b_scale, np.float64)[None, :]
    return y if row_bias is None else y + np.asarray(row_bias, np.float64)[:, None]
