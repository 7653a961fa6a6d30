"""Pins of the 4-bit rows' oracle: written-out values, the rule of the scale, the layout."""

import numpy as np
import pytest

from oracle.mx4 import LEVELS, matmul, pack, place, quantize, unpack, values


def _block(first, rest=0.0):
    z = np.full((1, 32), rest)
    z[0, :len(first)] = first
    return z


def test_grid_and_ties_to_the_even_code():
    # the largest element 6: scale 1
    z = _block([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.2500001, 0.7499999, 4.9999, 5.0001, -0.0])
    code, byte = quantize(z)
    assert byte[0, 0] == 127
    assert list(code[0, :14]) == [7, 0, 2, 2, 4, 4, 6, 6, 8, 9, 1, 6, 7, 8]
    assert np.array_equal(values(code, byte)[0, :3], [6.0, 0.0, 1.0])


@pytest.mark.parametrize("top,e", [(7.0, 0), (np.nextafter(7.0, 8.0), 1), (3.5, -1), (3.6, 0), (1.0, -2), (4.0, 0),
                                   (1e-45, -126), (2.0 ** -126 * 7, -126), (3.4e38, 126), (0.0, -126)])
def test_scale_is_the_smallest_that_holds_seven(top, e):
    code, byte = quantize(_block([top]))
    assert int(byte[0, 0]) - 127 == e
    assert top <= 7 * 2.0 ** e and (e == -126 or top > 7 * 2.0 ** (e - 1))


def test_error_is_at_most_half_the_step():
    rng = np.random.default_rng(0)
    z = (rng.standard_normal((64, 320)) * np.exp(rng.standard_normal((64, 320)))).astype(np.float32)
    code, byte = quantize(z)
    scale = np.repeat(np.exp2(byte.astype(np.float64) - 127), 32, axis=1)
    a = np.abs(z) / scale
    step = np.where(a < 2, 0.5, np.where(a < 4, 1.0, 2.0))
    assert (np.abs(values(code, byte) - z) <= step / 2 * scale).all()
    # a search over all levels finds none nearer
    best = np.abs(a[:, :, None] - LEVELS).min(axis=2) * scale
    assert np.array_equal(np.abs(values(code, byte) - z), best)


def test_blocks_that_are_not_finite():
    z = np.ones((1, 100))
    z[0, 40], z[0, 99] = np.inf, np.nan
    code, byte = quantize(z)
    assert list(byte[0]) == [125, 255, 125, 255]
    v = values(code, byte)
    assert np.isnan(v[0, 32:64]).all() and np.isnan(v[0, 96:]).all() and (v[0, :32] == 1).all() and (v[0, 64:96] == 1).all()
    assert not code[0, 32:64].any()


@pytest.mark.parametrize("cols", [1, 31, 33, 500, 512, 1027])
def test_layout(cols):
    rng = np.random.default_rng(cols)
    z = rng.standard_normal((3, cols))
    code, byte = quantize(z)
    q, scale = pack(code, byte, fill=0xEE)
    assert q.shape[1] % 16 == 0 and scale.shape[1] % 16 == 0
    c, b = unpack(q, scale, cols)
    assert np.array_equal(c, code) and np.array_equal(b, byte)
    if cols % 2:
        assert (q[:, cols // 2] >> 4 == 0).all()
    # sixteen blocks fill sixteen bytes, four consecutive blocks lie four bytes apart
    assert sorted(place(i) for i in range(32)) == list(range(32))
    assert [place(i) for i in (0, 1, 2, 3, 4, 5, 16)] == [0, 4, 8, 12, 1, 5, 16]


def test_product_of_values():
    rng = np.random.default_rng(1)
    a, b = rng.standard_normal((3, 70)), rng.standard_normal((5, 70))
    va, vb = values(*quantize(a), factor=[1, 2, 3]), values(*quantize(b))
    y = matmul(va, vb, [1, 2, 3])
    for i in range(3):
        for j in range(5):
            assert y[i, j] == pytest.approx(sum(va[i, k] * vb[j, k] for k in range(70)) + i + 1, rel=1e-12)
