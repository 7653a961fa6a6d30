"""The 4-bit product through k_mx4_tile: every end of the last group, ranges of K,
strided results, scales of NaN, rows far apart and results beyond the cache, for each
tile (the sizes and what they reach: mx4_plan.py).

References are float64 products on the GPU.  The elements' products are exact; each
addition inside and between the matrix instructions is off by at most 2 u (truncation)
of its result's size, u = 2^-24, so a sum of n terms is within 2 n u / (1 - 2 n u) of the
sum of the magnitudes, n = K + 32 (the joins of the ranges); the factors, the bias and
their products add 4 u, and one storage rounding comes last.  Sums of multiples of 1/4
below 2^22 are exact.
"""

import pytest

from gpu_util import torch_dtype
from mx4_plan import LARGE, SPLIT, UNSPLIT

pytestmark = pytest.mark.gpu

tw = pytest.importorskip("activation_sparse_transformer_bf16_amd")

U = 2.0 ** -24
US = {"f32": U, "bf16": 2.0 ** -8}
ONE = [s for cases in UNSPLIT.values() for s in cases]
CUT = list(SPLIT.values())
LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _places(cols):
    """Where the scale bytes of a row's blocks lie."""
    return [b // 16 * 16 + b % 4 * 4 + b // 4 % 4 for b in range((cols + 31) // 32)]


def _rows(rows, cols, g, spread=6):
    """Rows with scales of 2^-spread ... 2^spread, codes other than zero and scales of NaN
    behind their ends, and their values in float64."""
    import torch
    q = torch.randint(0, 256, (rows, (cols + 31) // 32 * 16), generator=g, device="cuda:0", dtype=torch.uint8)
    places = torch.tensor(_places(cols), device="cuda:0")
    byte = torch.randint(127 - spread, 128 + spread, (rows, len(places)), generator=g, device="cuda:0", dtype=torch.uint8)
    scale = torch.full((rows, (len(places) + 15) // 16 * 16), 255, dtype=torch.uint8, device="cuda:0")
    scale[:, places] = byte
    return tw.Mx4Rows(q[:, :(cols + 1) // 2], scale, cols), _values(q, byte, cols)


def _values(q, byte, cols):
    import torch
    level = torch.tensor(LEVELS + [-v for v in LEVELS], dtype=torch.float64, device="cuda:0")
    code = torch.stack([q & 15, q >> 4], 2).reshape(q.shape[0], -1)
    return (level[code.long()] * torch.exp2(byte.double() - 127).repeat_interleave(32, 1))[:, :cols].contiguous()


def _operands(M, N, K, seed, spread=6):
    import torch
    g = torch.Generator(device="cuda:0")
    g.manual_seed(seed)
    a, va = _rows(M, K, g, spread)
    b, vb = _rows(N, K, g, spread)
    fa = torch.rand(M, generator=g, device="cuda:0") + 0.01
    fb = (torch.rand(N, generator=g, device="cuda:0") + 0.01) / K ** 0.5
    return a, va, fa, b, vb, fb, torch.randn(M, generator=g, device="cuda:0")


def _matmul(va, vb):
    return va @ vb.t().contiguous()


def _check(y, va, vb, fa, fb, bias, dtype):
    f = 1.0 if fa is None else fa.double()[:, None] * fb.double()
    want, size = _matmul(va, vb) * f, _matmul(va.abs(), vb.abs()) * f
    if bias is not None:
        want, size = want + bias.double()[:, None], size + bias.double().abs()[:, None]
    n = va.shape[1] + 32
    bound = (2 * n * U / (1 - 2 * n * U) + 4 * U) * size
    bad = ~((y.double() - want).abs() <= bound + US[dtype] * (want.abs() + bound))
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} outside, first at {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", ONE + CUT)
def test_product(dtype, M, N, K):
    # plain, then with factors and bias into a y at odd offsets and an odd stride inside
    # a wider buffer: what lies around it stays as it was
    print(f"product {dtype} {M} x {N} x {K}", flush=True)
    import torch
    a, va, fa, b, vb, fb, bias = _operands(M, N, K, M + N + K)
    dt = torch_dtype(dtype)
    y = tw.twell_mx4_matmul(a, b, dtype=dt)
    _check(y, va, vb, None, None, None, dtype)
    assert torch.equal(y, tw.twell_mx4_matmul(a, b, dtype=dt))
    buf = torch.full((M + 2, (N + 21) | 1), 7.0, dtype=dt, device="cuda:0")
    y = buf[1:M + 1, 3:3 + N]
    assert y.stride(0) % 2 == 1
    assert tw.twell_mx4_matmul(a._replace(factor=fa), b._replace(factor=fb), row_bias=bias, y=y) is y
    _check(y, va, vb, fa, fb, bias, dtype)
    for part in (buf[0], buf[M + 1], buf[:, :3], buf[:, 3 + N:]):
        assert bool((part == 7).all())


@pytest.mark.parametrize("M,N,K", ONE + CUT)
def test_sums_of_quarters_are_exact(M, N, K):
    # scales of 1, 36 K < 2^22 (K < 116508); factors that are powers of two
    print(f"exact product {M} x {N} x {K}", flush=True)
    import torch
    a, va, _, b, vb, _, _ = _operands(M, N, K, M + N + K + 1, spread=0)
    fa, fb = torch.full((M,), 0.25, device="cuda:0"), torch.full((N,), 8.0, device="cuda:0")
    want = _matmul(va, vb).float()
    assert torch.equal(tw.twell_mx4_matmul(a, b, dtype=torch.float32), want)
    assert torch.equal(tw.twell_mx4_matmul(a._replace(factor=fa), b._replace(factor=fb), dtype=torch.float32), 2 * want)


@pytest.mark.parametrize("M,N,K", ONE + CUT)
def test_nan_scales(M, N, K):
    # a NaN scale of any block (the first, the last, one between) makes its row or column NaN
    # and no other value
    print(f"NaN scales {M} x {N} x {K}", flush=True)
    import torch
    a, _, _, b, _, _, _ = _operands(M, N, K, M + N + K + 2)
    y = tw.twell_mx4_matmul(a, b, dtype=torch.float32)
    place = _places(K)
    at = [place[0], place[-1], place[len(place) // 2]]
    rows, cols = [2, M - 1, M // 2], [0, N - 1, N // 3]
    a.scale[rows, at] = 255
    b.scale[cols, at] = 255
    z = tw.twell_mx4_matmul(a, b, dtype=torch.float32)
    assert bool(z[rows].isnan().all()) and bool(z[:, cols].isnan().all())
    y[rows] = float("nan")
    y[:, cols] = float("nan")
    assert torch.equal(z.isnan(), y.isnan()) and torch.equal(z.nan_to_num(0.0), y.nan_to_num(0.0))


@pytest.mark.parametrize("dtype,M,N,K", [(t, *s) for t in LARGE for s in LARGE[t]])
def test_large_results(dtype, M, N, K):
    print(f"large product {dtype} {M} x {N} x {K}", flush=True)
    a, va, fa, b, vb, fb, bias = _operands(M, N, K, M + N + K + 3)
    y = tw.twell_mx4_matmul(a._replace(factor=fa), b._replace(factor=fb), row_bias=bias, dtype=torch_dtype(dtype))
    _check(y, va, vb, fa, fb, bias, dtype)


@pytest.mark.parametrize("M,N,K,ld", [(8648, 445, 3599, 7864320), (5519, 643, 3137, 7864320), (8498, 386, 1212, 7864320),
                                      (8648, 445, 3599, 7864336), (6111, 142, 3645, 16777216), (20, 300, 700, 8388608)])
def test_rows_far_apart(M, N, K, ld):
    # 32-bit offsets within a tile up to rows 7864320 bytes apart, 64-bit ones beyond
    print(f"rows {ld} bytes apart, {M} x {N} x {K}", flush=True)
    import torch
    a, va, fa, b, vb, fb, _ = _operands(M, N, K, M + N + K + 4)
    wide = torch.empty(N, ld, dtype=torch.uint8, device="cuda:0")
    n = b.q.shape[1]
    wide[:, :(n + 15) // 16 * 16] = 0xFF
    wide[:, :n] = b.q
    far = tw.Mx4Rows(wide[:, :n], b.scale, K, fb)
    _check(tw.twell_mx4_matmul(a._replace(factor=fa), far, dtype=torch.float32), va, vb, fa, fb, None, "f32")
    swap = tw.twell_mx4_matmul(far, a._replace(factor=fa), dtype=torch.float32)
    _check(swap, vb, va, fb, fa, None, "f32")


def test_ranges_in_a_captured_graph_with_one_workspace():
    # three products in a row through the same workspace, replayed with other operands and
    # eager products through it in between
    import torch
    shapes = [SPLIT[128, 128, 4], SPLIT[64, 128, 16], SPLIT[256, 128, 2]]
    sets = [[_operands(M, N, K, 7 * i + seed) for i, (M, N, K) in enumerate(shapes)] for seed in (1, 2, 3)]
    now = [tuple(tw.Mx4Rows.empty(r.rows, r.cols, "cuda:0") for r in (o[0], o[3])) for o in sets[0]]
    workspace = torch.empty(max(tw.twell_mx4_matmul_workspace_size(*s) for s in shapes), dtype=torch.uint8, device="cuda:0")
    results = [torch.empty(M, N, device="cuda:0") for M, N, _ in shapes]

    def products(rows, ys):
        for (a, b), y in zip(rows, ys):
            tw.twell_mx4_matmul(a, b, y=y, workspace=workspace)

    def load(of):
        for to, o in zip(now, of):
            for dst, src in zip(to, (o[0], o[3])):
                # (what a view leaves out: the bytes up to the next multiple of 16, never read into a result)
                dst.q.copy_(src.q)
                dst.scale.copy_(src.scale)

    load(sets[0])
    products(now, results)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        products(now, results)
    for of in (sets[1], sets[2], sets[0]):
        load(of)
        for r in results:
            r.fill_(-1.0)
        graph.replay()
        got = [r.clone() for r in results]
        eager = [torch.empty_like(r) for r in results]
        products(now, eager)
        torch.cuda.synchronize()
        for g, e, o in zip(got, eager, of):
            assert torch.equal(g, e)
            _check(g, o[1], o[4], None, None, None, "f32")
