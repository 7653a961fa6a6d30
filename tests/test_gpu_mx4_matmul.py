"""GPU parity of the 4-bit product with the float64 oracle.

The elements' products are exact (multiples of 1/4 times a power of two); the sums
are fp32 in an order and precision inside the matrix instruction that no document
fixes.  Each addition is off by at most 2 u (truncation) of its result's size,
u = 2^-24, so a sum of n terms is within 2 n u / (1 - 2 n u) of the sum of the
magnitudes, n = K + 32 (the joins of up to 32 ranges); the factors, the bias and
their products add 4 u, and one storage rounding comes last.  Sums that fit 24
bits whole are exact.
"""

import numpy as np
import pytest

from oracle.mx4 import matmul, pack, values
from oracle.numerics import decode, round_to_storage

from gpu_util import assert_bitwise, from_dev, torch_dtype

pytestmark = pytest.mark.gpu

tw = pytest.importorskip("activation_sparse_transformer_bf16_amd")

U = 2.0 ** -24
US = {"f32": U, "bf16": 2.0 ** -8}


def make(rows, cols, seed, spread=6, mid=127):
    """(codes, scale bytes) with scales 2^-spread ... 2^spread round 2^(mid - 127)."""
    rng = np.random.default_rng(seed)
    code = rng.integers(0, 16, (rows, cols)).astype(np.uint8)
    byte = rng.integers(mid - spread, mid + spread + 1, (rows, -(-cols // 32))).astype(np.uint8)
    return code, byte


def dev(code, byte, factor=None, fill=0xFF):
    """On the GPU, with `fill` (codes of -6, scales NaN) behind every row's end."""
    import torch
    q, scale = pack(code, byte, fill=fill)
    cols = code.shape[1]
    if cols % 2:
        q[:, cols // 2] |= 0xF0  # the odd half of the last byte is not read either
    qd = torch.from_numpy(q).to("cuda:0")
    f = None if factor is None else torch.from_numpy(np.ascontiguousarray(factor, np.float32)).to("cuda:0")
    return tw.Mx4Rows(qd[:, :(cols + 1) // 2], torch.from_numpy(scale).to("cuda:0"), cols, f)


def vec(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to("cuda:0")


def check(y, a, b, fa, fb, bias, dtype):
    va, vb = values(*a), values(*b)
    K = va.shape[1]
    f = (1.0 if fa is None else fa[:, None].astype(np.float64)) * (1.0 if fb is None else fb[None, :].astype(np.float64))
    want = matmul(va, vb) * f
    size = matmul(np.abs(va), np.abs(vb)) * np.abs(f)
    if bias is not None:
        want = want + bias[:, None].astype(np.float64)
        size = size + np.abs(bias[:, None].astype(np.float64))
    n = K + 32
    bound = (2 * n * U / (1 - 2 * n * U) + 4 * U) * size
    got = decode(from_dev(y.contiguous(), dtype), dtype)
    err = np.abs(got - want)
    limit = bound + US[dtype] * (np.abs(want) + bound)
    bad = ~(err <= limit)
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[0]}"


# M, N, K: single elements; below, at and above every tile edge; K inside, at and
# just past blocks of 32, slabs of 128 and groups of 512; few rows with many columns and
# the other way round; few tiles with a long K
SHAPES = [(1, 1, 1), (1, 5, 3), (2, 16, 16), (1, 64, 64), (1, 1000, 777), (3, 257, 100), (7, 96, 2048), (16, 16, 128),
          (17, 33, 65), (31, 100, 255), (32, 128, 256), (33, 130, 257), (64, 64, 384), (65, 63, 512), (100, 300, 640),
          (127, 129, 767), (128, 128, 1024), (129, 257, 1280), (200, 1, 600), (255, 256, 127), (256, 256, 2048),
          (257, 511, 2061), (300, 700, 96), (333, 1000, 777), (513, 515, 800), (1, 2048, 8192), (8, 8192, 512),
          (48, 512, 4096), (64, 2048, 8192), (32, 300, 16384), (17, 131, 5003), (100, 1, 4096),
          (300, 260, 20000), (129, 1000, 7777), (700, 520, 2000), (1500, 300, 288), (1024, 1024, 1024),
          (2076, 18, 42), (122, 1133, 548), (440, 578, 1664), (257, 1996, 983), (101, 4171, 39), (4564, 391, 33),
          (4104, 928, 19), (2067, 1593, 150), (4, 6, 50556), (1, 1524, 24721), (2349, 39, 9705), (1637, 257, 8417),
          (17, 8603, 2438), (708, 394, 2092), (5157, 38, 2082)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(dtype, M, N, K):
    print(f"product {dtype} {M} x {N} x {K}", flush=True)
    rng = np.random.default_rng(M + N + K)
    a, b = make(M, K, 1), make(N, K, 2)
    fa = (rng.random(M) + 0.01).astype(np.float32)
    fb = ((rng.random(N) + 0.01) / np.sqrt(K)).astype(np.float32)
    bias = rng.standard_normal(M).astype(np.float32)
    t = torch_dtype(dtype)
    check(tw.twell_mx4_matmul(dev(*a), dev(*b), dtype=t), a, b, None, None, None, dtype)
    check(tw.twell_mx4_matmul(dev(*a, factor=fa), dev(*b, factor=fb), row_bias=vec(bias), dtype=t), a, b, fa, fb, bias,
          dtype)


@pytest.mark.parametrize("M,N,K", [(1, 33, 4096), (16, 48, 4096), (130, 70, 4096), (300, 260, 3001), (520, 513, 2047),
                                   (64, 64, 8000), (1030, 1000, 500)])
def test_small_sums_are_exact(M, N, K):
    # scales of 1 and 2: every sum is a multiple of 1/4 below 36 * 4 * 8000 < 2^21, 23 bits
    a, b = make(M, K, 3, spread=0), make(N, K, 4, spread=0)
    a = (a[0], a[1] + np.random.default_rng(0).integers(0, 2, a[1].shape).astype(np.uint8))
    b = (b[0], b[1] + np.random.default_rng(1).integers(0, 2, b[1].shape).astype(np.uint8))
    y = tw.twell_mx4_matmul(dev(*a), dev(*b), dtype=torch_dtype("f32"))
    assert_bitwise(y.cpu().numpy() + 0.0, matmul(values(*a), values(*b)).astype(np.float32) + 0.0, "y")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K,ld,off", [(5, 70, 100, 75, 3), (140, 130, 128, 131, 1), (300, 264, 64, 272, 8),
                                          (20, 64, 64, 200, 1), (600, 530, 256, 533, 3)])
def test_output_strides_and_input_views(dtype, M, N, K, ld, off):
    # y inside a wider buffer (what lies around it stays), operands as slices of wider rows
    import torch
    a, b = make(M, K, 6), make(N, K, 7)
    da, db = dev(*a), dev(*b)
    wide_q = torch.full((M, 512), 0xFF, dtype=torch.uint8, device="cuda:0")
    wide_s = torch.full((M, 96), 0xFF, dtype=torch.uint8, device="cuda:0")
    n = da.q.shape[1]
    wide_q[:, 32:32 + n] = da.q
    wide_s[:, 48:48 + da.scale.shape[1]] = da.scale
    av = tw.Mx4Rows(wide_q[:, 32:32 + n], wide_s[:, 48:48 + da.scale.shape[1]], K)
    y = torch.full((M, ld), 5.0, dtype=torch_dtype(dtype), device="cuda:0")
    tw.twell_mx4_matmul(av, db, y=y[:, off:off + N])
    check(y[:, off:off + N], a, b, None, None, None, dtype)
    assert (y[:, :off] == 5).all() and (y[:, off + N:] == 5).all()


@pytest.mark.parametrize("M,N", [(1, 40), (33, 50), (130, 140), (300, 520)])
def test_special_scales_and_factors(M, N):
    # NaN blocks reach their row or column and nothing else; infinite sums and factors
    K = 700
    a, b = make(M, K, 8), make(N, K, 9)
    a[1][M // 2, 3] = 255
    b[1][N // 3, 21] = 255
    fa = np.ones(M, np.float32)
    fa[0] = np.inf if M > 1 else 1.0
    y = tw.twell_mx4_matmul(dev(*a, factor=fa), dev(*b), dtype=torch_dtype("f32")).cpu().numpy()
    nan = np.zeros((M, N), bool)
    nan[M // 2], nan[:, N // 3] = True, True
    want = matmul(values(*a), values(*b))
    assert np.isnan(y[nan]).all()
    rest = ~nan
    rest[0] = False
    assert np.isfinite(y[rest]).all()
    size = matmul(np.abs(values(*a)), np.abs(values(*b)))
    n = K + 32
    assert (np.abs(y[rest] - want[rest]) <= (2 * n * U / (1 - 2 * n * U) + 4 * U) * size[rest] * (1 + U)).all()
    if M > 1:
        fine = ~nan[0] & (want[0] != 0)
        assert np.isinf(y[0][fine]).all() and (np.sign(y[0][fine]) == np.sign(want[0][fine])).all()


@pytest.mark.parametrize("mid_a,mid_b", [(7, 247), (40, 100), (30, 127), (200, 60)])
def test_far_scales(mid_a, mid_b):
    # products from subnormal fp32 numbers on; 2^-133 is far below the smallest step counted
    M, N, K = 40, 70, 300
    a, b = make(M, K, 10, mid=mid_a), make(N, K, 11, mid=mid_b)
    y = tw.twell_mx4_matmul(dev(*a), dev(*b), dtype=torch_dtype("f32")).cpu().numpy()
    va, vb = values(*a), values(*b)
    want, size = matmul(va, vb), matmul(np.abs(va), np.abs(vb))
    n = K + 32
    assert (np.abs(y - want) <= (2 * n * U / (1 - 2 * n * U) + 4 * U) * size + n * 2.0 ** -149).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N", [(0, 5), (5, 0), (0, 0)])
def test_empty(dtype, M, N):
    y = tw.twell_mx4_matmul(dev(*make(M, 64, 0)), dev(*make(N, 64, 0)), dtype=torch_dtype(dtype))
    assert y.shape == (M, N)


def test_same_result_again_and_on_another_stream():
    import torch
    a, b = make(300, 4096, 12), make(520, 4096, 13)
    da, db = dev(*a), dev(*b)
    y = tw.twell_mx4_matmul(da, db, dtype=torch.float32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = tw.twell_mx4_matmul(da, db, dtype=torch.float32)
    s.synchronize()
    assert torch.equal(y, again)


def test_binding_refuses():
    import torch
    a, b = dev(*make(3, 64, 0)), dev(*make(4, 64, 0))
    bad = [lambda: tw.twell_mx4_matmul(a, dev(*make(4, 96, 0))),
           lambda: tw.twell_mx4_matmul(a, b, row_bias=vec(np.zeros(4))),
           lambda: tw.twell_mx4_matmul(a, b, y=torch.empty(3, 5, dtype=torch.bfloat16, device="cuda:0")),
           lambda: tw.twell_mx4_matmul(a._replace(factor=vec(np.ones(2))), b),
           lambda: tw.twell_mx4_matmul(a._replace(scale=a.scale[:, :8]), b),
           lambda: tw.twell_mx4_matmul(a._replace(q=a.q[:, :31]), b),
           lambda: tw.twell_mx4_matmul(a._replace(q=torch.zeros(3, 40, dtype=torch.uint8, device="cuda:0")[:, :32]), b),
           # rows whose last 16-byte chunk is not there
           lambda: tw.twell_mx4_matmul(tw.Mx4Rows(torch.zeros(20, dtype=torch.uint8, device="cuda:0")[:20].view(1, 20),
                                                  torch.zeros(1, 16, dtype=torch.uint8, device="cuda:0"), 40),
                                       dev(*make(4, 40, 0)))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        tw.twell_mx4_matmul(a, b.q)  # not Mx4Rows
    with pytest.raises(TypeError):
        tw.twell_mx4_matmul(a, b, dtype=torch.float16)
