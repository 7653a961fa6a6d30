"""The feed-forward block of examples/ffn_block.py served with its gate in 8 bits
where some rows overflow the TwELL capacity: those take the dense fallback, whose
gate comes from the weights in the activations' type; the others keep the 8-bit
gate.  Tolerances as for the layer (gpu_util.TOL)."""

import numpy as np
import pytest

from oracle.block import int8_matmul, quantize_rows, residual_sum, rmsnorm, rmsnorm_quantized
from oracle.ffn import ffn, ffn_from_h, rel_l2
from oracle.numerics import decode, round_to_storage
from oracle.twell import relu_storage

from gpu_util import TOL, assert_bitwise, from_dev
from test_gpu_block import EPS, _block, _inputs

pytestmark = pytest.mark.gpu

tw = pytest.importorskip("activation_sparse_transformer_bf16_amd")


@pytest.mark.parametrize("dtype,T,d,F", [("f32", 67, 256, 512), ("bf16", 96, 512, 1024), ("bf16", 1, 512, 1024)])
@pytest.mark.parametrize("every", [1, 3])
def test_rows_that_overflow(dtype, T, d, F, every):
    tile, cap = 128, 16
    s = _inputs(T, d, F, dtype, 4)
    s["bias"][::every] = 1.0  # most units of these rows are active
    block, dev = _block(s, dtype, cap=cap, tile=tile)
    y, h = block.serve(dev["x"], dev["res"], dev["bias"])
    h_o = residual_sum(s["x"], s["res"], dtype)
    assert_bitwise(from_dev(h, dtype), h_o, "h")
    q, scale = rmsnorm_quantized(h_o, s["norm"], EPS, dtype)
    qw, sw = quantize_rows(s["wg"], dtype)
    act = relu_storage(round_to_storage(int8_matmul(q, scale, qw, sw, s["bias"]), dtype), dtype)
    n = round_to_storage(rmsnorm(h_o, s["norm"], EPS, dtype), dtype)
    over = (np.count_nonzero(decode(act, dtype).reshape(T, F // tile, tile) > 0, axis=2) > cap).any(axis=1)
    # the rows with the raised bias overflow, and no other: over 100 active units
    # a tile against at most 9
    assert np.array_equal(np.nonzero(over)[0], np.arange(0, T, every))
    want = ffn_from_h(decode(act, dtype), n, s["wu"], s["wd"], dtype)
    dense = ffn(n, s["wg"], s["wu"], s["wd"], s["bias"], dtype)
    got = decode(from_dev(y, dtype), dtype)
    assert rel_l2(got[over], dense[over]) <= TOL[dtype]
    if dtype == "f32":  # that is not the 8-bit gate, which bf16's rounding would hide
        assert rel_l2(want[over], dense[over]) > 100 * TOL[dtype]
    if (~over).any():
        assert rel_l2(got[~over], want[~over]) <= TOL[dtype]
