"""Rows of microscaled 4-bit floats and their product (oracle side).

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

Definitions (``include/twell.h``): blocks of 32 elements share 2^e, e the
smallest whole number in -126 ... 126 with max |z| <= 7 * 2^e; an element is the
nearest of LEVELS times 2^e (ties to the even code), its sign in bit 3 of the code.
A block with an infinite or NaN element: codes 0, scale byte 255.
"""

from __future__ import annotations

import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = 32


def place(b):
    """Where block b's scale byte lies in its row."""
    return b // 16 * 16 + b % 4 * 4 + b // 4 % 4


def blocks(z: np.ndarray) -> np.ndarray:
    """[rows, blocks, 32] with zeros behind the last column."""
    rows, cols = z.shape
    out = np.zeros((rows, -(-cols // BLOCK) * BLOCK))
    out[:, :cols] = z
    return out.reshape(rows, -1, BLOCK)


def quantize(z: np.ndarray):
    """(codes uint8 [rows, cols], scale bytes uint8 [rows, blocks]) of fp32 (or wider) rows."""
    rows, cols = z.shape
    z = blocks(np.asarray(z, np.float64))
    bad = ~np.isfinite(z).all(axis=2)
    z = np.where(bad[:, :, None], 0.0, z)
    top = np.abs(z).max(axis=2)
    # top / 7 = f 2^k with f in [0.5, 1): 2^(k-1) is enough only where f is 0.5
    f, k = np.frexp(top / 7.0)
    e = np.where(top == 0.0, -126, np.clip(np.where(f == 0.5, k - 1, k), -126, 126))
    a = np.abs(z) * np.exp2(-e.astype(np.float64))[:, :, None]
    code = np.zeros(a.shape, np.uint8)
    for i in range(1, 8):
        mid = (LEVELS[i - 1] + LEVELS[i]) / 2
        # a tie goes to the even one of codes i - 1 and i
        code = np.where((a > mid) | ((a == mid) & (i % 2 == 0)), np.uint8(i), code)
    code |= (np.signbit(z).astype(np.uint8) << 3).astype(np.uint8)
    code = np.where(bad[:, :, None], np.uint8(0), code)
    byte = np.where(bad, 255, e + 127).astype(np.uint8)
    return code.reshape(rows, -1)[:, :cols], byte


def values(code: np.ndarray, byte: np.ndarray, factor=None) -> np.ndarray:
    """What codes and scale bytes stand for, float64."""
    cols = code.shape[1]
    v = np.where(code >= 8, -1.0, 1.0) * LEVELS[code & 7]
    scale = np.where(byte == 255, np.nan, np.exp2(byte.astype(np.float64) - 127.0))
    out = v * np.repeat(scale, BLOCK, axis=1)[:, :cols]
    return out if factor is None else out * np.asarray(factor, np.float64)[:, None]


def pack(code: np.ndarray, byte: np.ndarray, fill: int = 0x5A):
    """(q [rows, 16 * ceil(cols / 32)], scale [rows, 16 * ceil(cols / 512)]) as the
    library lays them out, ``fill`` where no operator writes."""
    rows, cols = code.shape
    q = np.full((rows, -(-cols // 32) * 16), fill, np.uint8)
    even = np.zeros((rows, -(-cols // 2) * 2), np.uint8)
    even[:, :cols] = code
    q[:, :even.shape[1] // 2] = even[:, 0::2] | (even[:, 1::2] << 4)
    scale = np.full((rows, -(-cols // 512) * 16), fill, np.uint8)
    for b in range(byte.shape[1]):
        scale[:, place(b)] = byte[:, b]
    return q, scale


def unpack(q: np.ndarray, scale: np.ndarray, cols: int):
    """(codes, scale bytes) of rows as the library lays them out."""
    code = np.empty((q.shape[0], 2 * q.shape[1]), np.uint8)
    code[:, 0::2], code[:, 1::2] = q & 15, q >> 4
    return code[:, :cols], scale[:, [place(b) for b in range(-(-cols // BLOCK))]]


def matmul(a: np.ndarray, b: np.ndarray, row_bias=None) -> np.ndarray:
    """a b^T + bias of values, float64."""
    with np.errstate(all="ignore"):
        y = a @ b.T
    return y if row_bias is None else y + np.asarray(row_bias, np.float64)[:, None]
