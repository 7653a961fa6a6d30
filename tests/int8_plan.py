"""The 8-bit product's choice of kernel, tile and K ranges (i8_plan in
csrc/int8.hip), written once more with the constants read from the source, so
that tests can say which kernel a size pins.  test_int8_plan.py holds it to the
library's own choice."""

from __future__ import annotations

import os
import re

_SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                       "activation_sparse_transformer_bf16_amd", "csrc", "int8.hip")
with open(_SOURCE) as f:
    _TEXT = f.read()


def _constant(name: str) -> int:
    return int(re.search(rf"constexpr int {name} = (\d+);", _TEXT).group(1))


def _table(name: str):
    body = re.search(rf"{name}\[\w+\] = \{{(.*?)\}};", _TEXT, re.S).group(1)
    return [tuple(int(v) for v in row.split(",")) for row in re.findall(r"\{([\d, ]+)\}", body)]


TILES = _table("I8_COST")    # rows, columns, cost of a slab
SMALL = _table("I8_SMALL")   # rows, columns, workgroups a CU holds, start, round
TILE_COST, JOIN_COST, MAX_PARTS = _constant("I8_TILE_COST"), _constant("I8_JOIN_COST"), _constant("I8_MAX_PARTS")
SMALL_RATE = _constant("I8_SMALL_RATE")
MAX_PARTIAL = 64 << 20
SLAB = 64


def _up(a: int, b: int) -> int:
    return -(-a // b)


def plan(M: int, N: int, K: int):
    """(kernel "tile" or "small", rows, columns, K ranges, workspace bytes)."""
    nk, read = _up(K, SLAB), (M + N) * K
    best, least = None, None
    for bm, bn, held, start, rnd in SMALL:
        tiles = _up(M, bm) * _up(N, bn)
        cost = start + _up(tiles, 256 * held) * rnd + _up(tiles, 256) * ((bm + bn) * K // SMALL_RATE) + read // 140000
        if least is None or cost < least:
            best, least = ("small", bm, bn, 1, 0), cost
    for bm, bn, slab in TILES:
        tiles = _up(M, bm) * _up(N, bn)
        want = 1
        while want <= MAX_PARTS:
            per = _up(nk, want)
            parts = _up(nk, per)
            sums = parts * M * _up(N, 4) * 4
            if want > 1 and (parts < want or per < 4 or sums * 4 > MAX_PARTIAL):
                break
            cost = max(_up(tiles * parts, 256) * (per * slab + TILE_COST), read // 50000 + TILE_COST)
            cost += JOIN_COST + sums // 5000 if parts > 1 else 0
            if cost < least:
                best, least = ("tile", bm, bn, parts, sums * 4 if parts > 1 else 0), cost
            want *= 2
    return best


# Sizes that reach k_int8_tile, with ragged rows, columns and K (K over more
# slabs than the ring has stages): for each tile a product on one range of K, with
# few slabs and with many, ...
UNSPLIT = {(64, 128): [(66, 6865, 396), (1300, 1100, 9000)], (128, 128): [(8251, 133, 391), (2100, 1700, 5003)],
           (256, 128): [(8386, 391, 388), (2500, 2300, 3001)], (256, 256): [(822, 8297, 386), (5001, 4001, 1003)]}
# ... and products on each number of ranges.
SPLIT = {(64, 128, 2): (33, 8273, 16343), (64, 128, 4): (33, 4178, 10578), (64, 128, 8): (33, 1621, 17325),
         (64, 128, 16): (35, 33, 22100), (128, 128, 2): (8660, 67, 7764), (128, 128, 4): (65, 5571, 9417),
         (128, 128, 8): (2390, 34, 20986), (128, 128, 16): (400, 300, 65530), (256, 128, 2): (8301, 263, 22837),
         (256, 128, 4): (8417, 65, 8839), (256, 128, 8): (4461, 33, 24984), (256, 128, 16): (520, 513, 65535),
         (256, 256, 2): (513, 7339, 8961), (256, 256, 4): (197, 8278, 10488), (256, 256, 8): (1001, 1203, 65535),
         (256, 256, 16): (1001, 999, 65535)}
# Results beyond 256 MB (stored non-temporally), and whole prompt batches through
# the gates of the 1.5B-class and of the larger layer.
LARGE = {"f32": [(8201, 8203, 391)], "bf16": [(16401, 8203, 391), (8192, 8192, 2048), (16384, 14336, 4096)]}
