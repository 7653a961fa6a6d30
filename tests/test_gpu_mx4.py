"""GPU parity of the 4-bit rows with the oracle: the quantiser, the reader, the
norm that writes them.

Codes and scale bytes are matters of the input's bits and compared bit for bit.
A value read is an exact fp32 number (an element times a power of two), one fp32
product with the row's factor and one storage rounding.
"""

import numpy as np
import pytest

from oracle.block import norm_factor, residual_sum, rmsnorm
from oracle.mx4 import pack, place, quantize, unpack, values
from oracle.numerics import decode, round_to_storage

from gpu_util import assert_bitwise, from_dev, to_dev, torch_dtype

pytestmark = pytest.mark.gpu

tw = pytest.importorskip("activation_sparse_transformer_bf16_amd")

U = 2.0 ** -24
US = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
FILL = 0xC3

# single elements; below, at and past blocks of 32, chunks of a wave (256 and 512
# elements), groups of 512; many short rows, few long ones
SHAPES = [(1, 1), (1, 2), (3, 7), (5, 31), (64, 32), (7, 33), (2, 64), (33, 65), (300, 40), (4, 100), (9, 127),
          (17, 128), (5, 255), (6, 256), (3, 257), (2, 511), (7, 512), (3, 513), (1, 1000), (130, 1000), (65, 1027),
          (2, 2048), (3, 4100), (1, 16384), (2, 20001), (1000, 96), (2049, 17)]


def _rows(rows, cols, dtype, seed):
    rng = np.random.default_rng(seed)
    z = rng.standard_normal((rows, cols)) * np.exp(1.5 * rng.standard_normal((rows, cols)))
    z *= np.exp(4 * rng.standard_normal((rows, 1)))
    z[rng.random(z.shape) < 0.02] = 0.0
    # values on ties and levels
    tie = rng.choice([0.25, 0.5, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, -0.25, -0.75, -7.0], z.shape)
    z = np.where(rng.random(z.shape) < 0.1, tie, z)
    return round_to_storage(z, dtype) if dtype == "bf16" else z.astype(np.float32)


def _out(rows, cols, factor=False, extra=0):
    """Buffers filled with FILL, with rows `extra` * 16 bytes further apart than needed."""
    import torch
    ld, lds = -(-cols // 32) * 16 + 16 * extra, -(-cols // 512) * 16
    q = torch.full((rows, ld), FILL, dtype=torch.uint8, device="cuda:0")
    scale = torch.full((rows, lds + 16 * extra), FILL, dtype=torch.uint8, device="cuda:0")
    f = torch.zeros(rows, device="cuda:0") if factor else None
    return tw.Mx4Rows(q[:, :(cols + 1) // 2], scale[:, :lds], cols, f), q, scale


def _check_bits(q, scale, z, what):
    """The whole buffers against the oracle's, FILL where nothing may be written."""
    code, byte = quantize(z)
    want_q, want_scale = pack(code, byte, fill=FILL)
    wide_q = np.full(q.shape, FILL, np.uint8)
    wide_scale = np.full(scale.shape, FILL, np.uint8)
    wide_q[:, :want_q.shape[1]], wide_scale[:, :want_scale.shape[1]] = want_q, want_scale
    assert_bitwise(scale.cpu().numpy(), wide_scale, f"{what} scales")
    assert_bitwise(q.cpu().numpy(), wide_q, f"{what} codes")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize_and_read(dtype, rows, cols):
    print(f"quantise {dtype} {rows} x {cols}", flush=True)
    x = _rows(rows, cols, dtype, rows + cols)
    out, q, scale = _out(rows, cols)
    tw.twell_quantize_mx4(to_dev(x, dtype), out)
    _check_bits(q, scale, decode(x, dtype), "quantiser")
    code, byte = quantize(decode(x, dtype))
    for read in ("f32", "bf16"):
        # an element times a power of two has three significant bits: exact in either type
        got = from_dev(tw.twell_dequantize_mx4(out, torch_dtype(read)), read)
        assert np.array_equal(decode(got, read), values(code, byte))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols,ld,off,extra", [(100, 131, 3, 1), (512, 520, 8, 0), (511, 513, 1, 2), (1000, 1003, 1, 0),
                                               (64, 64, 0, 3), (7, 9, 1, 1)])
def test_strides_and_alignment(dtype, cols, ld, off, extra):
    import torch
    rows = 13
    wide = _rows(rows, ld + off, dtype, cols)
    xd = to_dev(wide, dtype)[:, off:off + cols]
    out, q, scale = _out(rows, cols, extra=extra)
    tw.twell_quantize_mx4(xd, out)
    z = decode(np.ascontiguousarray(wide[:, off:off + cols]), dtype)
    _check_bits(q, scale, z, "quantiser")
    y = torch.full((rows, ld + off), 7.0, dtype=torch_dtype(dtype), device="cuda:0")
    tw.twell_dequantize_mx4(out, y=y[:, off:off + cols])
    got = decode(from_dev(y, dtype), dtype)
    assert np.array_equal(got[:, off:off + cols], values(*quantize(z)))
    assert (got[:, :off] == 7).all() and (got[:, off + cols:] == 7).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_every_scale_and_special_values(dtype):
    # a block for each power of two that the type holds, with inf, NaN, zeros and both
    # kinds of zero among them
    e = np.arange(-149 if dtype == "f32" else -133, 128)
    rng = np.random.default_rng(3)
    z = np.exp2(e.astype(np.float64))[:, None] * rng.choice([0.0, 0.3, 0.7, 1.0, 1.2, 1.6, 1.75, 1.9, -1.0, -1.8], (e.size, 32))
    z[:, 0] = np.exp2(e.astype(np.float64)) * rng.choice([1.0, 1.5, 1.75, 1.875], e.size)
    special = np.ones((6, 32))
    special[0, 5], special[1, 0], special[2, 31], special[3, 1] = np.inf, -np.inf, np.nan, -0.0
    special[4] = 0.0
    special[5] = -0.0
    big = np.finfo(np.float32).max if dtype == "f32" else 3.38e38
    z = np.concatenate([z, special, np.full((1, 32), big)])
    x = round_to_storage(z, dtype) if dtype == "bf16" else z.astype(np.float32)
    # as rows of one block, and as one row of many
    for a in (x, x.reshape(1, -1)):
        out, q, scale = _out(*a.shape)
        tw.twell_quantize_mx4(to_dev(a, dtype), out)
        _check_bits(q, scale, decode(a, dtype), "quantiser")
        got = tw.twell_dequantize_mx4(out, torch_dtype("f32")).cpu().numpy()
        code, byte = quantize(decode(a, dtype))
        # the storage rounding: the largest numbers have 4 * 2^126 as their nearest value,
        # 2^128, which is infinite in fp32
        with np.errstate(over="ignore"):
            want = values(code, byte).astype(np.float32)
        assert np.isinf(want).any()
        assert np.array_equal(got, want, equal_nan=True)


def test_read_every_code_scale_and_factor():
    # scale bytes that the quantiser never writes (0, 254) among them
    rng = np.random.default_rng(4)
    rows, cols = 256, 544
    byte = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 17, 1)
    code = rng.integers(0, 16, (rows, cols)).astype(np.uint8)
    factor = (rng.standard_normal(rows) * 3).astype(np.float32)
    factor[7], factor[9], factor[11] = 0.0, np.inf, np.nan
    q, scale = pack(code, byte)
    import torch
    r = tw.Mx4Rows(torch.from_numpy(q).to("cuda:0")[:, :cols // 2], torch.from_numpy(scale).to("cuda:0"), cols,
                   torch.from_numpy(factor).to("cuda:0"))
    # an element times 2^e in fp32 (subnormal or infinite where that is), times the factor
    with np.errstate(all="ignore"):
        exact = values(code, byte).astype(np.float32)
        want = exact * factor[:, None]
    got = tw.twell_dequantize_mx4(r, torch_dtype("f32")).cpu().numpy()
    assert np.array_equal(got, want, equal_nan=True)
    got = from_dev(tw.twell_dequantize_mx4(r, torch_dtype("bf16")), "bf16")
    fine = np.isfinite(want)
    with np.errstate(all="ignore"):
        assert np.array_equal(got[fine], round_to_storage(want[fine].astype(np.float64), "bf16"))
    assert np.array_equal(np.isnan(decode(got, "bf16")), np.isnan(want))


def test_empty_and_row_slices():
    import torch
    for cols in (1, 100):
        out = tw.twell_quantize_mx4(torch.zeros(0, cols, dtype=torch.bfloat16, device="cuda:0"))
        assert out.q.shape == (0, (cols + 1) // 2)
        assert tw.twell_dequantize_mx4(out).shape == (0, cols)
    x = _rows(20, 700, "f32", 1)
    whole = tw.twell_quantize_mx4(to_dev(x, "f32"))
    part = tw.Mx4Rows(whole.q[5:9], whole.scale[5:9], 700)
    assert np.array_equal(tw.twell_dequantize_mx4(part, torch_dtype("f32")).cpu().numpy().astype(np.float64),
                          values(*quantize(x[5:9])))


def test_offsets_beyond_32_bits():
    # rows far apart: the last one starts past 2^32 bytes
    import torch
    rows, cols, ld = 3, 200, (1 << 30) + 24
    wide = torch.empty((rows - 1) * ld + cols, dtype=torch.float32, device="cuda:0")
    x = wide.as_strided((rows, cols), (ld, 1))
    z = _rows(rows, cols, "f32", 2)
    x.copy_(torch.from_numpy(z))
    out = tw.twell_quantize_mx4(x)
    assert_bitwise(tw.twell_dequantize_mx4(out, torch_dtype("f32")).cpu().numpy(), values(*quantize(z)).astype(np.float32), "x")
    y = wide.as_strided((rows, cols), (ld, 1), storage_offset=0)
    y.zero_()
    tw.twell_dequantize_mx4(out, y=y)
    assert np.array_equal(y.cpu().numpy().astype(np.float64), values(*quantize(z)))


def _norm_case(rows, d, dtype, seed, residual=True):
    rng = np.random.default_rng(seed)

    def rand(*shape, loc=0.0):
        v = loc + rng.standard_normal(shape)
        return round_to_storage(v, dtype) if dtype == "bf16" else v.astype(np.float32)

    return rand(rows, d), rand(rows, d) if residual else None, rand(d, loc=1.0)


def _check_norm(out, q, scale, x, res, w, dtype, eps=1e-6):
    h = residual_sum(x, res, dtype)
    H = decode(h, dtype)
    z = (H.astype(np.float32) * decode(w, dtype).astype(np.float32)).astype(np.float32)
    _check_bits(q, scale, z, "norm")
    if res is not None and out.h is not None:
        assert_bitwise(from_dev(out.h, dtype), h, "h")
    # r: the squares' sum of d terms, a division, an addition and a reciprocal root of
    # 2 ulp: (d + 20) u relative at most (all terms are positive)
    r = norm_factor(h, eps, dtype)
    bound = (x.shape[1] + 20) * U
    assert (np.abs(out.q.factor.cpu().numpy() - r) <= bound * r).all()
    if out.y is not None:
        y = rmsnorm(h, w, eps, dtype)
        got = decode(from_dev(out.y, dtype), dtype)
        assert (np.abs(got - y) <= (bound + 4 * U + US[dtype] * (1 + bound + 4 * U)) * np.abs(y) + 2.0 ** -133).all()


# each split of a row over waves and lanes, whole rows and rows of no alignment
NORMS = [(1, 1), (3, 5), (2, 32), (5, 100), (1, 256), (7, 512), (4, 1000), (9, 1024), (2, 1031), (33, 2048), (3, 2050),
         (5, 4096), (2, 4099), (3, 8192), (1, 10001), (2, 16384), (1, 20000), (1, 32768)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,d", NORMS)
def test_norm(dtype, rows, d):
    print(f"norm {dtype} {rows} x {d}", flush=True)
    for residual in (True, False):
        x, res, w = _norm_case(rows, d, dtype, rows + d, residual)
        out, q, scale = _out(rows, d, factor=True)
        got = tw.twell_rmsnorm_mx4(to_dev(x, dtype), to_dev(w, dtype), 1e-6, None if res is None else to_dev(res, dtype),
                                   q=out)
        _check_norm(got, q, scale, x, res, w, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_longest_bf16_rows_and_forms(dtype):
    import torch
    d = 65536 if dtype == "bf16" else 32768
    x, res, w = _norm_case(2, d, dtype, 9)
    out, q, scale = _out(2, d, factor=True)
    xd, rd, wd = to_dev(x, dtype), to_dev(res, dtype), to_dev(w, dtype)
    _check_norm(tw.twell_rmsnorm_mx4(xd, wd, residual=rd, q=out), q, scale, x, res, w, dtype)
    # 4 bits alone; h and y over the inputs; the same bits as the two operators by themselves
    x, res, w = _norm_case(19, 1500, dtype, 10)
    xd, rd, wd = to_dev(x, dtype), to_dev(res, dtype), to_dev(w, dtype)
    out, q, scale = _out(19, 1500, factor=True)
    only = tw.twell_rmsnorm_mx4(xd, wd, residual=rd, q=out, want_y=False)
    assert only.y is None
    _check_norm(only, q, scale, x, res, w, dtype)
    plain = tw.twell_rmsnorm(xd, wd, residual=rd)
    out, q, scale = _out(19, 1500, factor=True)
    over = tw.twell_rmsnorm_mx4(xd, wd, residual=rd, h=rd, y=xd, q=out)
    assert over.h is rd and over.y is xd
    _check_norm(over, q, scale, x, res, w, dtype)
    assert torch.equal(over.y, plain.y) and torch.equal(over.h, plain.h)


def test_norm_special_rows():
    # a row with inf, one with NaN, one of zeros (eps = 0 and not), weights of zero
    x, _, w = _norm_case(5, 100, "f32", 11, False)
    x[0, 70], x[1, 3], x[2] = np.inf, np.nan, 0.0
    w[10:20] = 0.0
    for eps in (1e-6, 0.0):
        out, q, scale = _out(5, 100, factor=True)
        got = tw.twell_rmsnorm_mx4(to_dev(x, "f32"), to_dev(w, "f32"), eps, q=out)
        z = (x * w[None, :]).astype(np.float32)
        _check_bits(q, scale, z, "norm")
        r = got.q.factor.cpu().numpy()
        assert r[0] == 0 and np.isnan(r[1]) and (r[2] == (np.inf if eps == 0 else np.float32(1e3)) or abs(r[2] / 1e3 - 1) < 4 * U)


def test_places():
    assert sorted(place(np.arange(64))) == list(range(64))
    c, b = unpack(*pack(np.zeros((1, 600), np.uint8), np.arange(19, dtype=np.uint8)[None]), 600)
    assert list(b[0]) == list(range(19)) and not c.any()
