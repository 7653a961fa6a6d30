"""The 8-bit product through k_int8_tile: the ring's steady loop followed by the
scaled results, ranges of K, strided results, scales of NaN and results beyond
the cache, for each tile (the sizes and what they reach: int8_plan.py).

References are float64 products on the GPU, in which the integer sums are exact.
A result is (float(sum) * sa) * sb + bias: the conversion, the two products and
the addition carry at most 4 u = 2^-22 of |sum sa sb| + |bias|, then comes one
storage rounding.  With scales that are powers of two and sums below 2^24 only
the addition of the bias rounds, and fp32 results are compared bit for bit.
"""

import pytest

from gpu_util import torch_dtype
from int8_plan import LARGE, SPLIT, UNSPLIT

pytestmark = pytest.mark.gpu

tw = pytest.importorskip("activation_sparse_transformer_bf16_amd")

U = 2.0 ** -24
US = {"f32": U, "bf16": 2.0 ** -8}
ONE = [s for cases in UNSPLIT.values() for s in cases]
CUT = list(SPLIT.values())


def _rows(rows, cols, g, top=127, fill=99):
    """16-byte aligned int8 rows with something else than zero behind each."""
    import torch
    buf = torch.full((rows, (cols + 15) // 16 * 16), fill, dtype=torch.int8, device="cuda:0")
    buf[:, :cols] = torch.randint(-top, top + 1, (rows, cols), generator=g, device="cuda:0", dtype=torch.int8)
    return buf[:, :cols]


def _operands(M, N, K, seed, top=127):
    import torch
    g = torch.Generator(device="cuda:0")
    g.manual_seed(seed)
    a, b = _rows(M, K, g, top), _rows(N, K, g, top, fill=-77)
    sa = torch.rand(M, generator=g, device="cuda:0") + 0.01
    sb = (torch.rand(N, generator=g, device="cuda:0") + 0.01) / K ** 0.5
    return g, a, sa, b, sb, torch.randn(M, generator=g, device="cuda:0")


def _sums(a, b):
    """The integer sums in float64."""
    return a.double() @ b.double().t().contiguous()


def _check(y, sums, sa, sb, bias, dtype):
    part = sums * sa.double()[:, None] * sb.double()
    want = part if bias is None else part + bias.double()[:, None]
    bound = 4 * U * (part.abs() if bias is None else part.abs() + bias.double().abs()[:, None])
    bad = ~((y.double() - want).abs() <= bound + US[dtype] * (want.abs() + bound))
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} outside, first at {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", ONE + CUT)
def test_product(dtype, M, N, K):
    print(f"product {dtype} {M} x {N} x {K}", flush=True)
    import torch
    _, a, sa, b, sb, bias = _operands(M, N, K, M + N + K)
    sums = _sums(a, b)
    dt = torch_dtype(dtype)
    y = tw.twell_int8_matmul(a, sa, b, sb, dtype=dt)
    _check(y, sums, sa, sb, None, dtype)
    again = tw.twell_int8_matmul(a, sa, b, sb, dtype=dt)
    assert torch.equal(y, again)
    _check(tw.twell_int8_matmul(a, sa, b, sb, row_bias=bias, dtype=dt), sums, sa, sb, bias, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", ONE + CUT)
def test_strided_results(dtype, M, N, K):
    # y at odd offsets and an odd stride inside a wider buffer: what lies around
    # it stays as it was
    print(f"strided product {dtype} {M} x {N} x {K}", flush=True)
    import torch
    _, a, sa, b, sb, bias = _operands(M, N, K, M + N + K + 1)
    buf = torch.full((M + 2, (N + 21) | 1), 7.0, dtype=torch_dtype(dtype), device="cuda:0")
    y = buf[1:M + 1, 3:3 + N]
    assert y.stride(0) % 2 == 1
    assert tw.twell_int8_matmul(a, sa, b, sb, row_bias=bias, y=y) is y
    _check(y, _sums(a, b), sa, sb, bias, dtype)
    for part in (buf[0], buf[M + 1], buf[:, :3], buf[:, 3 + N:]):
        assert bool((part == 7).all())


@pytest.mark.parametrize("M,N,K", ONE + CUT)
def test_nan_scales(M, N, K):
    # a NaN scale makes its row or column NaN and no other value
    print(f"NaN scales {M} x {N} x {K}", flush=True)
    import torch
    _, a, sa, b, sb, _ = _operands(M, N, K, M + N + K + 2)
    y = tw.twell_int8_matmul(a, sa, b, sb, dtype=torch.float32)
    rows, cols = [2, M - 1], [0, N - 1]
    sa[rows], sb[cols] = float("nan"), float("nan")
    z = tw.twell_int8_matmul(a, sa, b, sb, dtype=torch.float32)
    assert bool(z[rows].isnan().all()) and bool(z[:, cols].isnan().all())
    y[rows] = float("nan")
    y[:, cols] = float("nan")
    assert torch.equal(z.isnan(), y.isnan()) and torch.equal(z.nan_to_num(0.0), y.nan_to_num(0.0))


@pytest.mark.parametrize("M,N,K", ONE + CUT)
def test_powers_of_two_are_exact(M, N, K):
    # sums of at most 65536 * 9 < 2^24
    print(f"exact product {M} x {N} x {K}", flush=True)
    import torch
    g, a, _, b, _, _ = _operands(M, N, K, M + N + K + 3, top=3)
    sa = 2.0 ** torch.randint(-3, 4, (M,), generator=g, device="cuda:0").float()
    sb = 2.0 ** torch.randint(-3, 4, (N,), generator=g, device="cuda:0").float()
    bias = torch.randint(-64, 65, (M,), generator=g, device="cuda:0") / 64.0
    want = _sums(a, b) * sa.double()[:, None] * sb.double() + bias.double()[:, None]
    assert torch.equal(tw.twell_int8_matmul(a, sa, b, sb, row_bias=bias, dtype=torch.float32), want.float())


@pytest.mark.parametrize("M,N,K", [UNSPLIT[t][1] for t in UNSPLIT] + [SPLIT[t] for t in SPLIT if t[2] in (2, 16)])
def test_largest_sums_are_exact(M, N, K):
    # -128 throughout a row of both, sums up to 2^30; unit scales, fp32 results:
    # the sum's own rounding to fp32 and nothing else
    print(f"largest sums {M} x {N} x {K}", flush=True)
    import torch
    _, a, _, b, _, _ = _operands(M, N, K, M + N + K + 4)
    a[M - 1], b[N - 1] = -128, -128
    one = lambda n: torch.ones(n, device="cuda:0")  # noqa: E731
    y = tw.twell_int8_matmul(a, one(M), b, one(N), dtype=torch.float32)
    assert torch.equal(y, _sums(a, b).float()) and float(y[M - 1, N - 1]) == 16384.0 * K


@pytest.mark.parametrize("dtype,M,N,K", [(t, *s) for t in LARGE for s in LARGE[t]])
def test_large_results(dtype, M, N, K):
    print(f"large product {dtype} {M} x {N} x {K}", flush=True)
    _, a, sa, b, sb, bias = _operands(M, N, K, M + N + K + 5)
    y = tw.twell_int8_matmul(a, sa, b, sb, row_bias=bias, dtype=torch_dtype(dtype))
    _check(y, _sums(a, b), sa, sb, bias, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tile", UNSPLIT, ids=str)
def test_operands_inside_wider_rows(dtype, tile):
    import torch
    M, N, K = UNSPLIT[tile][0]
    _, a, sa, b, sb, _ = _operands(M, N, K, 6)
    wa = torch.full((M, 32 + K // 16 * 16 + 80), 91, dtype=torch.int8, device="cuda:0")
    wb = torch.full((N, 16 + K // 16 * 16 + 16), -93, dtype=torch.int8, device="cuda:0")
    av, bv = wa[:, 32:32 + K], wb[:, 16:16 + K]
    av.copy_(a)
    bv.copy_(b)
    _check(tw.twell_int8_matmul(av, sa, bv, sb, dtype=torch_dtype(dtype)), _sums(a, b), sa, sb, None, dtype)
