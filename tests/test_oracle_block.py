"""Pins for the oracle's block operators (CPU only)."""

from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle.block import (int8_matmul, norm_factor, quantize, quantize_rows, residual_sum, rmsnorm,
                          rmsnorm_backward, rmsnorm_quantized)
from oracle.numerics import decode
from workloads.synth import to_storage

DTYPES = ["f32", "bf16"]


def _rand(shape, dtype, seed, spread=1.0):
    rng = np.random.default_rng(seed)
    return to_storage(rng.standard_normal(shape) * spread, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
def test_norm_hand_values(dtype):
    # mean square of (3, 4, 0, 0) is 25/4; eps 0: r = 2/5
    h = to_storage(np.array([[3.0, 4.0, 0.0, 0.0], [-2.0, 2.0, 2.0, -2.0]]), dtype)
    w = to_storage(np.array([1.0, 0.5, 2.0, 4.0]), dtype)
    assert np.allclose(rmsnorm(h, w, 0.0, dtype), [[1.2, 0.8, 0, 0], [-1.0, 0.5, 2.0, -4.0]], rtol=1e-15)
    # eps takes part in the mean square: 4 + 12 = 16
    assert np.allclose(norm_factor(h, 12.0, dtype)[1], 0.25, rtol=1e-15)


def test_residual_sum_rounds_once_to_storage():
    one = to_storage(np.array([[1.0, 1.0, 1.0]]), "bf16")
    add = to_storage(np.array([[2.0 ** -8, 3 * 2.0 ** -8, 2.0 ** -20]]), "bf16")
    # bf16 quantum at 1 is 2^-7: the first is a tie (to even), the second rounds up
    assert np.array_equal(decode(residual_sum(one, add, "bf16"), "bf16"), [[1.0, 1.0 + 2.0 ** -6, 1.0]])
    x = np.array([[1.0]], np.float32)
    assert residual_sum(x, None, "f32") is x


def test_quantize_hand_values_and_ties():
    z = np.array([[127.0, -127.0, 0.5, 1.5, -0.5, 2.5, 126.4]], np.float32)
    q, scale = quantize(z, np.ones(1))
    assert q.tolist() == [[127, -127, 0, 2, 0, 2, 126]] and scale[0] == 1.0
    # the row's factor reaches the scale only
    q2, scale2 = quantize(z, np.array([0.25]))
    assert np.array_equal(q, q2) and scale2[0] == 0.25
    zero, s0 = quantize(np.zeros((1, 3), np.float32), np.ones(1))
    assert not zero.any() and s0[0] == 2.0 ** -100 / 127.0
    bad, sb = quantize(np.array([[1.0, np.inf], [np.nan, 1.0], [1.0, 2.0]], np.float32), np.ones(3))
    assert not bad[:2].any() and np.isnan(sb[:2]).all() and bad[2].tolist() == [64, 127]


@pytest.mark.parametrize("dtype", DTYPES)
def test_quantized_rows_are_within_half_a_step(dtype):
    h, w = _rand((9, 65), dtype, 1, 3.0), _rand(65, dtype, 2)
    q, scale = rmsnorm_quantized(h, w, 1e-6, dtype)
    y = rmsnorm(h, w, 1e-6, dtype)
    assert np.all(np.abs(q * scale[:, None] - y) <= 0.5 * scale[:, None] * (1 + 2.0 ** -15))
    assert np.all(np.max(np.abs(q.astype(int)), axis=1) == 127)
    q, scale = quantize_rows(h, dtype)
    assert np.all(np.abs(q * scale[:, None] - decode(h, dtype)) <= 0.5 * scale[:, None] * (1 + 2.0 ** -15))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("with_dh", [False, True])
def test_gradient_equals_autograd_and_differences(dtype, with_dh):
    T, d, eps = 5, 11, 1e-3
    h, w, dy = _rand((T, d), dtype, 3), _rand(d, dtype, 4), _rand((T, d), dtype, 5)
    dh = _rand((T, d), dtype, 6) if with_dh else None
    dx, dw = rmsnorm_backward(dy, h, w, eps, dtype, dh)
    H = torch.tensor(decode(h, dtype), requires_grad=True)
    Wt = torch.tensor(decode(w, dtype), requires_grad=True)
    loss = (H / (H.pow(2).mean(1, keepdim=True) + eps).sqrt() * Wt * torch.tensor(decode(dy, dtype))).sum()
    if with_dh:
        loss = loss + (H * torch.tensor(decode(dh, dtype))).sum()
    loss.backward()
    assert np.allclose(dx, H.grad.numpy(), rtol=1e-12, atol=1e-13)
    assert np.allclose(dw, Wt.grad.numpy(), rtol=1e-12, atol=1e-13)

    def value(Hn, wn):
        y = Hn / np.sqrt(np.mean(Hn * Hn, axis=1, keepdims=True) + eps) * wn
        return np.sum(y * decode(dy, dtype)) + (0.0 if dh is None else np.sum(Hn * decode(dh, dtype)))

    Hn, wn, step = decode(h, dtype), decode(w, dtype), 1e-5
    for t, j in [(0, 0), (2, 7), (4, 10)]:
        up, down = Hn.copy(), Hn.copy()
        up[t, j] += step
        down[t, j] -= step
        assert abs((value(up, wn) - value(down, wn)) / (2 * step) - dx[t, j]) <= 1e-8 * max(1, abs(dx[t, j]))
    up, down = wn.copy(), wn.copy()
    up[3] += step
    down[3] -= step
    assert abs((value(Hn, up) - value(Hn, down)) / (2 * step) - dw[3]) <= 1e-8 * max(1, abs(dw[3]))


def test_gradient_is_orthogonal_without_eps():
    # y does not change along h when eps = 0: <dx, h> = 0
    h, w, dy = _rand((4, 33), "f32", 7), _rand(33, "f32", 8), _rand((4, 33), "f32", 9)
    dx, _ = rmsnorm_backward(dy, h, w, 0.0, "f32")
    assert np.max(np.abs(np.sum(dx * decode(h, "f32"), axis=1))) <= 1e-13


def test_product_equals_exact_rationals():
    rng = np.random.default_rng(10)
    a, b = rng.integers(-128, 128, (3, 7)).astype(np.int8), rng.integers(-128, 128, (4, 7)).astype(np.int8)
    sa, sb, bias = rng.random(3).astype(np.float32), rng.random(4).astype(np.float32), rng.random(3).astype(np.float32)
    y = int8_matmul(a, sa, b, sb, bias)
    for m in range(3):
        for n in range(4):
            s = sum(int(a[m, k]) * int(b[n, k]) for k in range(7))
            want = Fraction(s) * Fraction(float(sa[m])) * Fraction(float(sb[n])) + Fraction(float(bias[m]))
            assert abs(y[m, n] - float(want)) <= 1e-14 * max(1.0, abs(float(want)))
