"""AdamW with states in 32 or in microscaled 8 bits (oracle side).

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

Definitions (``include/twell.h``).  m and v are formed in fp32 with one rounding
per operation, which is part of the definition; the weights in float64.
"""

from __future__ import annotations

import numpy as np

BLOCK = 32
M32 = 0xFFFFFFFF


def mix(x: int) -> int:
    x ^= x >> 16
    x = x * 0x9E3779B1 & M32
    x ^= x >> 15
    x = x * 0x85EBCA6B & M32
    return x ^ (x >> 16)


def random_bits(seed: int, place: int, n: int) -> np.ndarray:
    """32 random bits per element: m takes the low 16, v the high 16, a bf16 weight the middle ones."""
    lo, hi = seed & M32, (seed >> 32) & M32
    key = mix((mix(lo ^ mix(hi)) + place) & M32)
    out = np.empty(n, np.uint32)
    for g in range(-(-n // 8)):
        base = mix(((g & M32) + key + (g >> 32) * 0x9E3779B1) & M32)
        for k in range(min(8, n - 8 * g)):
            x = (base + k * 0x9E3779B9) * 0x85EBCA6B & M32
            out[8 * g + k] = x ^ (x >> 16)
    return out


def encode(x: np.ndarray, random16: np.ndarray, fields: int):
    """(codes uint8 [n], scale bytes uint8) of fp32 x: 16 exponent fields with a sign
    (m) or 32 without (v)."""
    n = x.size
    nb = -(-n // BLOCK)
    a = np.zeros(nb * BLOCK)
    a[:n] = np.abs(x.astype(np.float64))
    a = a.reshape(nb, BLOCK)
    byte = np.empty(nb, np.uint8)
    code = np.zeros(nb * BLOCK, np.uint8)
    for b in range(nb):
        top = a[b].max()
        if not np.isfinite(a[b]).all() or top > 1.875 * 2.0 ** 113:
            byte[b] = 255
            continue
        e = -87
        while top > 1.875 * 2.0 ** e:
            e += 1
        byte[b] = e + 127
        for i in range(BLOCK):
            at = b * BLOCK + i
            if at >= n:
                break
            # the lowest exponent (fields 0 and 1 alike) has eight steps per power of two
            low = e - (fields - 2)
            k = max(int(np.floor(np.log2(a[b, i]))) if a[b, i] > 0 else low, low)
            part = int(np.floor(a[b, i] / 2.0 ** (k - 3) + (int(random16[at]) + 0.5) / 65536))
            c = (k - low) * 8 + part
            if fields == 32 and a[b, i] > 0:
                c = max(c, 1)
            code[at] = c | (128 if fields == 16 and np.signbit(x[at]) else 0)
    return code[:n], byte


def decode(code: np.ndarray, byte: np.ndarray, fields: int) -> np.ndarray:
    """The values, float64."""
    c = code.astype(np.int64) & (fields * 8 - 1)
    field = np.maximum(c >> 3, 1)
    part = np.where(c < 8, c, (c & 7) + 8)
    e = np.repeat(np.maximum(byte.astype(np.int64), 40), BLOCK)[:code.size] - 127
    v = part * np.exp2((e - (fields - 1) + field - 3).astype(np.float64))
    v = np.where(np.repeat(byte > 240, BLOCK)[:code.size], np.nan, v)
    return np.where(code.astype(np.int64) >= fields * 8, -v, v)


def moments(m, v, grad, beta1: float, beta2: float, factor=None):
    """(m, v) after the step, fp32, one rounding per operation."""
    f = np.float32
    with np.errstate(all="ignore"):
        g = np.asarray(grad, f) * f(1.0 if factor is None else factor)
        m = np.asarray(m, f) * f(beta1) + g * f(1.0 - beta1)
        v = np.asarray(v, f) * f(beta2) + (g * f(1.0 - beta2)) * g
    return m.astype(f), v.astype(f)


def weights(w, m, v, lr: float, step: int, beta1: float, beta2: float, eps: float, decay: float) -> np.ndarray:
    """w after the step from the new m and v, float64."""
    w, m, v = (np.asarray(t, np.float64) for t in (w, m, v))
    c1, c2 = 1.0 - beta1 ** step, 1.0 - beta2 ** step
    with np.errstate(all="ignore"):
        return (1.0 - lr * decay) * w - lr / c1 * m / (np.sqrt(v / c2) + eps)


def round_randomly(w: np.ndarray, random: np.ndarray) -> np.ndarray:
    """fp32 w to bf16 bits by the middle 16 of 32 random bits."""
    bits = np.ascontiguousarray(w, np.float32).view(np.uint32)
    return ((bits + ((random >> 8) & 0xFFFF)) >> 16).astype(np.uint16)


def grad_norm(grads, max_norm: float):
    """(norm, factor) in float64."""
    norm = float(np.sqrt(sum(float(np.sum(np.square(np.asarray(g, np.float64)))) for g in grads)))
    if not np.isfinite(norm) or norm > np.finfo(np.float32).max:
        return norm, float("nan")
    return norm, min(1.0, max_norm / norm) if norm > 0 else 1.0
