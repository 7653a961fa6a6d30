"""The sizes of the 4-bit product's tests reach the kernels they are meant for
(CPU only)."""

import numpy as np
import pytest

from mx4_plan import GROUP, LARGE, MAX_PARTIAL, SMALL, SPLIT, TILES, UNSPLIT, plan

tw = pytest.importorskip("activation_sparse_transformer_bf16_amd")


def test_plan_is_the_librarys():
    # the workspace is one [M][N] matrix of sums for each range of K, so its size
    # gives the library's choice wherever K is cut
    rng = np.random.default_rng(1)
    n_cut = 0
    for _ in range(20000):
        M, N = (int(np.exp(rng.uniform(0, np.log(20000)))) for _ in range(2))
        K = int(np.exp(rng.uniform(0, np.log(1 << 20))))
        size = plan(M, N, K)[4]
        assert tw.twell_mx4_matmul_workspace_size(M, N, K) == size <= MAX_PARTIAL, (M, N, K)
        n_cut += size > 0
    assert n_cut > 500


@pytest.mark.parametrize("tile", TILES, ids=str)
def test_tile_sizes(tile):
    bm, bn = tile[:2]
    ends = set()
    for M, N, K in UNSPLIT[bm, bn]:
        assert plan(M, N, K)[:4] == ("tile", bm, bn, 1), (M, N, K)
        assert M > bm and N > bn and M % bm and N % bn
        ends.add(((K - 1) % GROUP // 128, (K - 1) // GROUP % 2))
    assert len({slab for slab, _ in ends}) == 4 and {parity for _, parity in ends} == {0, 1}
    for parts in (2, 4, 8, 16):
        if (bm, bn) != (256, 256):  # takes all of K
            M, N, K = SPLIT[bm, bn, parts]
            assert plan(M, N, K)[:4] == ("tile", bm, bn, parts), (M, N, K)


def test_large_sizes():
    for dtype, cases in LARGE.items():
        for M, N, K in cases:
            assert plan(M, N, K)[:4] == ("tile", 256, 256, 1) and K > 2 * GROUP
    assert all(M * N * (2 if t == "bf16" else 4) > 256 << 20 for t, c in LARGE.items() for M, N, _ in c[:1])


def test_small_shapes_are_among_the_products_tested():
    from test_gpu_mx4_matmul import SHAPES
    assert {plan(*s)[1:3] for s in SHAPES if plan(*s)[0] == "small"} == {s[:2] for s in SMALL}
