"""GPU parity of the 8-bit product with the float64 oracle.

The integer sums are exact.  A result is (float(sum) * sa) * sb + bias: the
conversion, the two products and the addition carry at most 4 u = 2^-22 of
|sum sa sb| + |bias|, then comes one storage rounding.  With scales and biases
that are powers of two every step is exact and the fp32 result is compared bit
for bit.
"""

import numpy as np
import pytest

from oracle.block import int8_matmul
from oracle.numerics import decode, round_to_storage

from gpu_util import assert_bitwise, from_dev, torch_dtype

pytestmark = pytest.mark.gpu

tw = pytest.importorskip("activation_sparse_transformer_bf16_amd")

U = 2.0 ** -24
US = {"f32": U, "bf16": 2.0 ** -8}


def _int8(rows, cols, seed, extreme=False):
    rng = np.random.default_rng(seed)
    if extreme:
        return rng.choice(np.array([-128, -127, 127, 0, 1], np.int8), (rows, cols))
    return np.clip(np.rint(rng.standard_normal((rows, cols)) * 35), -127, 127).astype(np.int8)


def _dev(a, fill=99):
    """16-byte aligned int8 rows with something else than zero behind each row."""
    import torch
    rows, cols = a.shape
    buf = torch.full((rows, (cols + 15) // 16 * 16), fill, dtype=torch.int8, device="cuda:0")
    view = buf[:, :cols]
    view.copy_(torch.from_numpy(a))
    return view


def _vec(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to("cuda:0")


def _check(y, a, sa, b, sb, bias, dtype):
    want = int8_matmul(a, sa, b, sb, bias)
    size = np.abs(want if bias is None else want - bias[:, None].astype(np.float64)) + (
        0.0 if bias is None else np.abs(bias[:, None].astype(np.float64)))
    bound = 4 * U * size
    got = decode(from_dev(y.contiguous(), dtype), dtype)
    err = np.abs(got - want)
    limit = bound + US[dtype] * (np.abs(want) + bound)
    bad = ~(err <= limit)
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[0]}"


# M, N, K: single elements; below, at and above every tile edge; K inside,
# at and just past 16-byte chunks and 64-byte slabs; few rows with many columns
# and the other way round; few tiles with a long K (cut into ranges)
SHAPES = [(1, 1, 1), (1, 5, 3), (2, 16, 16), (1, 64, 64), (1, 1000, 777), (3, 257, 100), (7, 96, 2048), (16, 16, 64),
          (17, 33, 65), (31, 100, 127), (32, 128, 128), (33, 130, 129), (64, 64, 192), (65, 63, 256), (100, 300, 320),
          (127, 129, 383), (128, 128, 512), (129, 257, 640), (200, 1, 300), (255, 256, 63), (256, 256, 1024),
          (257, 511, 1031), (300, 700, 48), (333, 1000, 777), (513, 515, 400), (1, 2048, 8192), (8, 8192, 512),
          (48, 512, 4096), (64, 2048, 8192), (32, 300, 16384), (17, 131, 5003), (100, 1, 4096),
          (300, 260, 20000), (129, 1000, 7777), (700, 520, 2000), (1500, 300, 144), (1024, 1024, 1024),
          (2076, 18, 42), (122, 1133, 548), (440, 578, 832), (257, 1996, 983), (101, 4171, 39), (4564, 391, 33),
          (4104, 928, 19), (2067, 3593, 150), (4, 6, 50556), (1, 1524, 24721), (2349, 39, 29705), (1637, 257, 28417)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(dtype, M, N, K):
    print(f"product {dtype} {M} x {N} x {K}", flush=True)
    rng = np.random.default_rng(M + N + K)
    a, b = _int8(M, K, 1), _int8(N, K, 2)
    sa, sb = rng.random(M, np.float32) + 0.01, (rng.random(N, np.float32) + 0.01) / np.float32(np.sqrt(K))
    bias = rng.standard_normal(M).astype(np.float32)
    ad, bd = _dev(a), _dev(b, fill=-77)
    _check(tw.twell_int8_matmul(ad, _vec(sa), bd, _vec(sb), dtype=torch_dtype(dtype)), a, sa, b, sb, None, dtype)
    _check(tw.twell_int8_matmul(ad, _vec(sa), bd, _vec(sb), row_bias=_vec(bias), dtype=torch_dtype(dtype)), a, sa, b,
           sb, bias, dtype)


@pytest.mark.parametrize("M,N,K", [(1, 33, 65536), (16, 48, 65536), (130, 70, 65536), (300, 260, 5000), (520, 513, 65535)])
def test_sums_are_exact(M, N, K):
    # the largest magnitudes (-128 among them): sums up to 2^30; unit scales,
    # fp32 results: the sum's own rounding to fp32 and nothing else
    a, b = _int8(M, K, 3, True), _int8(N, K, 4, True)
    a[0], b[0] = -128, -128
    one = lambda n: _vec(np.ones(n))  # noqa: E731
    y = tw.twell_int8_matmul(_dev(a), one(M), _dev(b), one(N), dtype=torch_dtype("f32"))
    want = int8_matmul(a, np.ones(M), b, np.ones(N)).astype(np.float32)
    assert_bitwise(y.cpu().numpy(), want, "y")
    assert want[0, 0] == np.float32(16384.0 * K)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(1, 40, 96), (40, 72, 200), (200, 130, 100), (700, 600, 160)])
def test_powers_of_two_are_exact(dtype, M, N, K):
    rng = np.random.default_rng(5)
    a, b = rng.integers(-8, 9, (M, K)).astype(np.int8), rng.integers(-8, 9, (N, K)).astype(np.int8)
    sa, sb = 2.0 ** rng.integers(-3, 4, M), 2.0 ** rng.integers(-3, 4, N)
    bias = rng.integers(-64, 65, M) / 64.0
    y = tw.twell_int8_matmul(_dev(a), _vec(sa), _dev(b), _vec(sb), row_bias=_vec(bias), dtype=torch_dtype(dtype))
    assert_bitwise(from_dev(y, dtype), round_to_storage(int8_matmul(a, sa, b, sb, bias), dtype), "y")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K,ld,off", [(5, 70, 100, 75, 3), (140, 130, 128, 131, 1), (300, 264, 64, 272, 8), (20, 64, 64, 200, 1)])
def test_output_strides_and_input_views(dtype, M, N, K, ld, off):
    # y inside a wider buffer (what lies around it stays), operands as column
    # slices of wider rows
    import torch
    a, b = _int8(M, K, 6), _int8(N, K, 7)
    wide_a = torch.full((M, 512), 91, dtype=torch.int8, device="cuda:0")
    wide_b = torch.full((N, 1024), -93, dtype=torch.int8, device="cuda:0")
    av, bv = wide_a[:, 32:32 + K], wide_b[:, 1024 - (K + 15) // 16 * 16:][:, :K]
    av.copy_(torch.from_numpy(a))
    bv.copy_(torch.from_numpy(b))
    sa, sb = np.full(M, 0.5, np.float32), np.full(N, 0.25, np.float32)
    buf = torch.full((M, ld + 16), 7.0, dtype=torch_dtype(dtype), device="cuda:0")
    y = buf[:, off:off + N]
    assert tw.twell_int8_matmul(av, _vec(sa), bv, _vec(sb), y=y) is y
    _check(y, a, sa, b, sb, None, dtype)
    assert bool((buf[:, :off] == 7).all()) and bool((buf[:, off + N:] == 7).all())


@pytest.mark.parametrize("M", [4, 100, 600])
def test_special_scales(M):
    # a NaN scale (the quantiser's mark of a row with an infinity or NaN) makes
    # its row or column NaN and no other
    a, b = _int8(M, 64, 8), _int8(150, 64, 9)
    sa, sb = np.ones(M, np.float32), np.ones(150, np.float32)
    sa[2], sb[149] = np.nan, np.nan
    y = tw.twell_int8_matmul(_dev(a), _vec(sa), _dev(b), _vec(sb), dtype=torch_dtype("f32")).cpu().numpy()
    want = int8_matmul(a, sa, b, sb).astype(np.float32)
    assert np.array_equal(np.isnan(y), np.isnan(want)) and np.isnan(y[2]).all() and np.isnan(y[:, 149]).all()
    assert np.array_equal(y[~np.isnan(want)], want[~np.isnan(want)])


@pytest.mark.parametrize("K", [200, 50556])
def test_operands_beyond_32_bit_offsets(K):
    # rows 2^31 + 64 bytes apart: far outside 32-bit offsets from the first
    import torch
    ld = (1 << 31) + 64
    for M in (3, 20):
        a, b = _int8(M, K, 10), _int8(3, K, 11)
        wide = torch.empty(2 * ld + (1 << 16), dtype=torch.int8, device="cuda:0")
        bv = wide.as_strided((3, K), (ld, 1))
        bv.copy_(torch.from_numpy(b))
        sa, sb = np.ones(M, np.float32), np.ones(3, np.float32)
        _check(tw.twell_int8_matmul(_dev(a), _vec(sa), bv, _vec(sb), dtype=torch_dtype("f32")), a, sa, b, sb, None, "f32")
        # and as the left operand
        _check(tw.twell_int8_matmul(bv, _vec(sb), _dev(a), _vec(sa), dtype=torch_dtype("f32")), b, sb, a, sa, None, "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_results_beyond_the_cache(dtype):
    # over 256 MB of results, in rows of no alignment: sums below 2^24, so that
    # the fp32 product of the same whole numbers is exact
    import torch
    M, N, K = (8200, 16401, 48) if dtype == "bf16" else (4100, 16401, 48)
    a, b = _dev(_int8(M, K, 19)), _dev(_int8(N, K, 20))
    one = lambda n: torch.ones(n, device="cuda:0")  # noqa: E731
    y = tw.twell_int8_matmul(a, one(M), b, one(N), dtype=torch_dtype(dtype))
    assert y.numel() * y.element_size() > 256 << 20
    assert torch.equal(y, (a.float() @ b.float().t()).to(y.dtype))


def test_output_beyond_32_bit_offsets():
    # y rows 2^31 elements apart
    import torch
    M, N, K = 3, 200, 96
    a, b = _int8(M, K, 12), _int8(N, K, 13)
    ld = (1 << 31) + 8
    buf = torch.empty(2 * ld + 512, dtype=torch.bfloat16, device="cuda:0")
    y = buf.as_strided((M, N), (ld, 1))
    tw.twell_int8_matmul(_dev(a), _vec(np.ones(M)), _dev(b), _vec(np.ones(N)), y=y)
    _check(y, a, np.ones(M, np.float32), b, np.ones(N, np.float32), None, "bf16")


def test_cut_products_repeat_and_take_a_workspace():
    # K cut into ranges: the same bits again, over a workspace of any contents
    import torch
    M, N, K = 40, 515, 40000
    a, b = _int8(M, K, 17), _int8(N, K, 18)
    sa, sb = np.full(M, 0.5, np.float32), np.full(N, 0.125, np.float32)
    n = tw.twell_int8_matmul_workspace_size(M, N, K)
    assert n > 0
    args = (_dev(a), _vec(sa), _dev(b), _vec(sb))
    ws = torch.full((n + 256,), 85, dtype=torch.uint8, device="cuda:0")
    y = tw.twell_int8_matmul(*args, dtype=torch.float32, workspace=ws)
    assert bool((ws[n:] == 85).all())
    _check(y, a, sa, b, sb, None, "f32")
    again = tw.twell_int8_matmul(*args, dtype=torch.float32)
    assert_bitwise(again.cpu().numpy(), y.cpu().numpy(), "y of a second run")


def test_empty_and_another_stream():
    import torch
    a, b = _int8(70, 130, 14), _int8(40, 130, 15)
    none = tw.twell_int8_matmul(_dev(a)[:0], _vec(np.ones(0)), _dev(b), _vec(np.ones(40)))
    assert none.shape == (0, 40)
    none = tw.twell_int8_matmul(_dev(a), _vec(np.ones(70)), _dev(b)[:0], _vec(np.ones(0)))
    assert none.shape == (70, 0)
    ad, bd, sa, sb = _dev(a), _dev(b), _vec(np.full(70, 0.5)), _vec(np.full(40, 0.5))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = tw.twell_int8_matmul(ad, sa, bd, sb)
    s.synchronize()
    _check(y, a, np.full(70, 0.5, np.float32), b, np.full(40, 0.5, np.float32), None, "bf16")


def test_quantised_product_of_a_layer():
    # the norm's 8 bits times quantised weights stay within the two
    # quantisations' half steps of the fp32 product
    import torch
    T, d, F = 96, 512, 640
    g = torch.Generator(device="cuda:0")
    g.manual_seed(16)
    x = torch.randn(T, d, generator=g, device="cuda:0").bfloat16()
    w = torch.ones(d, device="cuda:0").bfloat16()
    wg = (torch.randn(F, d, generator=g, device="cuda:0") / d ** 0.5).bfloat16()
    n = tw.twell_rmsnorm(x, w, 1e-6, quantize=True)
    qw, sw = tw.twell_quantize_rows(wg)
    y = tw.twell_int8_matmul(n.q, n.scale, qw, sw, dtype=torch.float32).cpu().double()
    yf, wf = n.y.float().cpu().double(), wg.float().cpu().double()
    sx, sw64 = n.scale.cpu().double()[:, None], sw.cpu().double()[:, None]
    # |dx| <= sx/2 + 2^-8 |y|, |dw| <= sw/2 per element
    dx, dw = 0.5 * sx + 2.0 ** -8 * yf.abs(), 0.5 * sw64
    bound = dx @ wf.abs().t() + (yf.abs() + dx) @ dw.expand(F, d).t()
    assert bool(((y - yf @ wf.t()).abs() <= bound * 1.0001).all())


def test_refusals():
    import torch
    q = torch.zeros(4, 64, dtype=torch.int8, device="cuda:0")
    s = torch.ones(4, device="cuda:0")
    with pytest.raises(ValueError):
        tw.twell_int8_matmul(q, s, q[:, :48], s)             # different K
    with pytest.raises(TypeError):
        tw.twell_int8_matmul(q.float(), s, q, s)
    with pytest.raises(TypeError):
        tw.twell_int8_matmul(q, s.double(), q, s)
    with pytest.raises(ValueError):
        tw.twell_int8_matmul(q, s[:3], q, s)
    with pytest.raises(ValueError):
        tw.twell_int8_matmul(q.t(), torch.ones(64, device="cuda:0"), q, s)
    with pytest.raises(ValueError):
        tw.twell_int8_matmul(q[:, :60].contiguous(), s, q[:, :60], s)    # rows of 60 bytes: not 16-byte aligned
    with pytest.raises(ValueError):
        # the last row's chunk would end outside the storage
        tw.twell_int8_matmul(torch.zeros(3 * 64 + 60, dtype=torch.int8, device="cuda:0").as_strided((4, 60), (64, 1)), s, q[:, :60], s)
    with pytest.raises(tw.TwellError):
        tw.twell_int8_matmul(q[:, 8:40], s, q[:, 8:40], s)   # base not 16-byte aligned
    with pytest.raises(TypeError):
        tw.twell_int8_matmul(q, s, q, s, dtype=torch.float16)
