"""Pins of the optimiser's oracle: torch's AdamW in float64, the 8-bit codes, the random rounding."""

import numpy as np
import pytest

from oracle.adamw import decode, encode, grad_norm, mix, moments, random_bits, round_randomly, weights


def test_step_is_adamw():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(0)
    w0 = rng.standard_normal(50)
    p = torch.nn.Parameter(torch.from_numpy(w0.copy()))
    opt = torch.optim.AdamW([p], lr=1e-2, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
    w, m, v = w0, np.zeros(50), np.zeros(50)
    for t in range(1, 6):
        g = rng.standard_normal(50).astype(np.float32)
        p.grad = torch.from_numpy(g.astype(np.float64))
        opt.step()
        m, v = moments(m, v, g, 0.9, 0.95)
        w = weights(w, m, v, 1e-2, t, 0.9, 0.95, 1e-8, 0.1)
    # m and v are fp32 here: a few 2^-24 in five steps of about 1e-2 each
    assert np.abs(w - p.detach().numpy()).max() < 5 * 1e-2 * 8 * 2.0 ** -24


@pytest.mark.parametrize("fields", [16, 32])
def test_every_code_is_kept(fields):
    # a block whose largest value fixes the scale, and every code in turn
    half = np.full(32, 0x8000, np.uint32)
    for byte in (40, 127, 200, 240):
        for c in range(256):
            code = np.zeros(32, np.uint8)
            code[0], code[1] = fields * 8 - 1, c
            x = decode(code, np.array([byte], np.uint8), fields)
            back, scale = encode(x, half, fields)
            assert scale[0] == byte and (back[1] & (fields * 8 - 1)) == (c & (fields * 8 - 1))
            assert back[1] == c or x[1] == 0


def test_code_values():
    one = np.array([127], np.uint8)
    v = lambda c, f: decode(np.array([c], np.uint8), one, f)[0]  # noqa: E731
    assert v(127, 16) == 1.875 and v(255, 16) == -1.875 and v(120, 16) == 1.0
    assert v(8, 16) == 2.0 ** -14 and v(7, 16) == 0.875 * 2.0 ** -14 and v(1, 16) == 2.0 ** -17 and v(0, 16) == 0
    assert v(255, 32) == 1.875 and v(8, 32) == 2.0 ** -30 and v(1, 32) == 2.0 ** -33
    assert decode(np.array([120], np.uint8), np.array([0], np.uint8), 16)[0] == 2.0 ** -87
    assert np.isnan(decode(np.array([0], np.uint8), np.array([241], np.uint8), 16)[0])


@pytest.mark.parametrize("fields", [16, 32])
@pytest.mark.parametrize("x", [1.0, 1.01, 1.99, 0.3, 3.3e-4, 2.0 ** -15 * 1.1, 2.0 ** -16 * 0.77])
def test_rounding_is_right_in_the_mean(fields, x):
    x = np.float32(x)
    at = np.arange(0, 65536, 17, dtype=np.uint32)
    got = []
    for i in range(0, at.size, 31):
        r = np.zeros(32, np.uint32)
        n = min(31, at.size - i)
        r[1:n + 1] = at[i:i + n]
        block = np.full(32, x, np.float32)
        block[0] = 1.875
        code, byte = encode(block, r, fields)
        got.append(decode(code, byte, fields)[1:n + 1])
    got = np.concatenate(got)
    # the dithers are a grid of spacing 17 / 65536 of a step: the mean is as near, and each value a neighbour
    step = max(2.0 ** (np.floor(np.log2(float(x))) - 3), 2.0 ** -17 if fields == 16 else 2.0 ** -33)
    assert abs(got.mean() - float(x)) <= 2 * step * 17 / 65536
    assert (np.abs(got - float(x)) < step).all()


def test_positive_v_stays_positive():
    x = np.full(32, 1e-30, np.float32)
    x[0] = 1.0
    code, byte = encode(x, np.zeros(32, np.uint32), 32)
    assert (code[1:] == 1).all()
    code, byte = encode(x, np.zeros(32, np.uint32), 16)
    assert (code[1:] == 0).all()


def test_blocks_that_are_not_finite():
    x = np.ones(70, np.float32)
    x[40], x[69] = np.nan, np.inf
    code, byte = encode(x, np.zeros(70, np.uint32), 16)
    assert list(byte) == [127, 255, 255]
    assert np.isnan(decode(code, byte, 16)[32:]).all()


def test_random_bits():
    a, b, c = random_bits(5, 0, 4096), random_bits(5, 1, 4096), random_bits(6, 0, 4096)
    for x in (a, b, c):
        # 16 bits each half: the mean of 4096 uniform numbers is within 6 / sqrt(12 * 4096) of one half
        for part in (x & 0xFFFF, x >> 16, (x >> 8) & 0xFFFF):
            assert abs((part / 65536).mean() - 0.5) < 6 / np.sqrt(12 * 4096)
    for x, y in ((a, b), (a, c), (b, c)):
        assert (x == y).mean() < 0.01
    assert np.array_equal(random_bits(5, 0, 100), a[:100])
    assert not np.array_equal(random_bits(5 + (1 << 32), 0, 100), a[:100])


def test_weights_rounded_randomly():
    w = np.full(4096, np.float32(1.0 + 2.0 ** -8 + 2.0 ** -9), np.float32)  # three quarters up of the step 2^-7
    got = round_randomly(w, random_bits(1, 0, 4096)).astype(np.uint32) << 16
    got = got.view(np.float32)
    assert set(np.unique(got)) == {np.float32(1.0), np.float32(1.0 + 2.0 ** -7)}
    assert abs((got > 1).mean() - 0.75) < 6 * np.sqrt(0.75 * 0.25 / 4096)


def test_grad_norm():
    assert grad_norm([[3.0], [4.0]], 1.0) == (5.0, 0.2)
    assert grad_norm([[3.0], [4.0]], 10.0) == (5.0, 1.0)
    assert grad_norm([[0.0]], 1.0) == (0.0, 1.0)
    assert np.isnan(grad_norm([[np.inf]], 1.0)[1])


@pytest.mark.parametrize("fields,smallest", [(16, 2.0 ** -104), (32, 2.0 ** -120)])
def test_bf16_holds_every_state(fields, smallest):
    # at most 4 significant bits, from `smallest` (a normal number) on
    code, byte = np.tile(np.arange(256, dtype=np.uint8), 241), np.repeat(np.arange(241, dtype=np.uint8), 8)
    v = decode(code, byte, fields)
    assert np.array_equal((v.astype(np.float32).view(np.uint32) & 0xFFFF0000).view(np.float32).astype(np.float64), v)
    assert np.abs(v[v != 0]).min() == smallest
