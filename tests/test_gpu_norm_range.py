"""The RMS norm and its gradient at the ends of their range: rows whose squares'
sum passes 2^128 while their mean square does not, beside ordinary rows and
within one row, in every split of a row over lanes and waves; rows beyond the
range; eps of zero.

The sums of such rows are taken of terms scaled by a power of two, which rounds
nothing, so the tolerances are those of test_gpu_norm.py: y and scale within 55
u, dx within 270 u and dweight within (T + 120) u of their absolute terms.  The
gradient's h r carries r's 51 u and one rounding, its r mean(g h) at most 51 +
90 + 10: together below the 270 u as before.
"""

import numpy as np
import pytest

from oracle.block import rmsnorm, rmsnorm_backward, rmsnorm_quantized
from oracle.numerics import decode
from workloads.synth import to_storage

from gpu_util import assert_bitwise, from_dev, to_dev
from test_gpu_norm import U, _close, _weight

pytestmark = pytest.mark.gpu

tw = pytest.importorskip("activation_sparse_transformer_bf16_amd")

# Row lengths for one to sixteen waves a row and one to eight chunks a lane, with
# rows shorter than a chunk, and rows that are whole chunks or not.
LENGTHS = {"f32": [3, 200, 301, 512, 777, 1024, 2048, 2049, 4096, 8192, 16384, 16401, 32768],
           "bf16": [7, 304, 511, 1024, 2048, 2049, 4096, 8192, 8195, 16384, 32768, 65528]}
CASES = [(t, d) for t in ("f32", "bf16") for d in LENGTHS[t]]


def _rows(d, sizes, T, seed):
    """T rows in turn of each kind in `sizes`: a size, or (size, size of its last quarter, size of its last value)."""
    rng = np.random.default_rng(seed)
    v = np.clip(rng.standard_normal((T, d)), -3.5, 3.5)
    # no value near zero: a quotient by it would say nothing
    v = np.where(np.abs(v) < 0.01, 0.01, v)
    for t in range(T):
        k = sizes[t % len(sizes)]
        if isinstance(k, tuple):
            v[t, :d - d // 4] *= 2.0 ** k[0]
            v[t, d - d // 4:] *= 2.0 ** k[1]
            v[t, -1] = 2.0 ** k[2]
        else:
            v[t] *= 2.0 ** k
    return v


# mean squares up to 2^126 (their sums up to 2^142), parts of a row of different
# sizes, and one large value in an ordinary row
HIGH = [0, 50, 56, 60, 62, 63, (45, 52, 50), (62, 60, 45), (0, 0, 63), 1]
# without eps to speak of: mean squares down to 2^-120
LOW = [0, -40, -50, -55, -59, (-50, -58, -52), (-58, -31, -31), (-100, -100, 0), (0, 0, 55), 1]


def _check(dtype, d, sizes, eps, T, seed):
    print(f"{dtype} {T} x {d} eps {eps}", flush=True)
    h, w = to_storage(_rows(d, sizes, T, seed), dtype), _weight(d, dtype, seed + 1)
    hd, wd = to_dev(h, dtype), to_dev(w, dtype)
    out = tw.twell_rmsnorm(hd, wd, eps, quantize=True)
    y64 = rmsnorm(h, w, eps, dtype)
    assert np.isfinite(y64).all() and np.abs(y64).max() > 0.1
    _close(decode(from_dev(out.y, dtype), dtype), y64, 55 * U * np.abs(y64), dtype, "y")
    q, scale = rmsnorm_quantized(h, w, eps, dtype)
    assert_bitwise(out.q.cpu().numpy(), q, "q")
    assert np.all(np.abs(out.scale.cpu().numpy().astype(np.float64) - scale) <= 55 * U * scale)
    dy = to_storage(np.random.default_rng(seed + 2).standard_normal((T, d)), dtype)
    dx, dw = tw.twell_rmsnorm_backward(to_dev(dy, dtype), hd, wd, eps)
    dx64, dw64 = rmsnorm_backward(dy, h, w, eps, dtype)
    H, DY, W = decode(h, dtype), decode(dy, dtype), decode(w, dtype)
    r = 1.0 / np.sqrt(np.mean(H * H, axis=1, keepdims=True) + eps)
    g = np.abs(DY * W)
    bound = 270 * U * (r * g + r * np.abs(H * r) * np.mean(g * np.abs(H * r), axis=1, keepdims=True))
    _close(decode(from_dev(dx, dtype), dtype), dx64, bound, dtype, "dx")
    assert np.all(np.abs(dw.cpu().numpy() - dw64) <= (T + 120) * U * np.sum(np.abs(DY * H) * r, axis=0))


@pytest.mark.parametrize("dtype,d", CASES)
def test_large_rows(dtype, d):
    _check(dtype, d, HIGH, 1e-6, 23, 41)


@pytest.mark.parametrize("dtype,d", CASES)
@pytest.mark.parametrize("eps", [0.0, 2.0 ** -140])
def test_small_rows_without_eps(dtype, d, eps):
    _check(dtype, d, LOW, eps, 23, 44)


@pytest.mark.parametrize("dtype,d", CASES)
def test_small_rows_beside_an_ordinary_eps(dtype, d):
    _check(dtype, d, [0, -30, -60, -75, -100, -110, (-100, -100, 0), (0, -100, -100)], 1e-6, 11, 47)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [5, 300, 2048, 8200])
def test_rows_beyond_the_range(dtype, d):
    # a mean square of 2^128 or more counts as infinite: r = 0, so y and scale are
    # zeros and dx is dh; rows beside it are as ever
    v = _rows(d, [0, 70, 100, 62], 8, 55)
    h, w = to_storage(v, dtype), _weight(d, dtype, 56)
    out = tw.twell_rmsnorm(to_dev(h, dtype), to_dev(w, dtype), 1e-6, quantize=True)
    y, scale = decode(from_dev(out.y, dtype), dtype), out.scale.cpu().numpy()
    far, near = [1, 2, 5, 6], [0, 3, 4, 7]
    assert not y[far].any() and not scale[far].any()
    y64 = rmsnorm(h, w, 1e-6, dtype)[near]
    _close(y[near], y64, 55 * U * np.abs(y64), dtype, "y")
    dy, dh = (to_storage(np.random.default_rng(k).standard_normal((8, d)), dtype) for k in (57, 58))
    dx, dw = tw.twell_rmsnorm_backward(to_dev(dy, dtype), to_dev(h, dtype), to_dev(w, dtype), 1e-6, to_dev(dh, dtype))
    assert_bitwise(from_dev(dx, dtype)[far], dh[far], "dx of rows beyond the range")
    _, dw64 = rmsnorm_backward(dy[near], h[near], w, 1e-6, dtype)
    r = 1.0 / np.sqrt(np.mean(decode(h[near], dtype) ** 2, axis=1, keepdims=True) + 1e-6)
    terms = np.sum(np.abs(decode(dy[near], dtype) * decode(h[near], dtype)) * r, axis=0)
    assert np.all(np.abs(dw.cpu().numpy() - dw64) <= (8 + 120) * U * terms)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [5, 300, 2048, 8200])
def test_zero_rows(dtype, d):
    # 1 / sqrt(0 + 0) is infinite: a row of zeros is NaN without eps, and zeros
    # with the smallest; the rows beside it are untouched
    v = _rows(d, [0, 0, -50], 6, 50)
    v[1] = 0.0
    h, w = to_storage(v, dtype), _weight(d, dtype, 51)
    others = [0, 2, 3, 4, 5]
    for eps in (0.0, 2.0 ** -149):
        out = tw.twell_rmsnorm(to_dev(h, dtype), to_dev(w, dtype), eps, quantize=True)
        y, scale = decode(from_dev(out.y, dtype), dtype), out.scale.cpu().numpy()
        assert not out.q.cpu().numpy()[1].any()
        if eps == 0.0:
            assert np.isnan(y[1]).all() and not np.isfinite(scale[1])
        else:
            assert not y[1].any() and np.isfinite(scale[1])
        y64 = rmsnorm(h, w, eps, dtype)[others]
        _close(y[others], y64, 55 * U * np.abs(y64), dtype, "y")
        dy = to_storage(np.random.default_rng(52).standard_normal((6, d)), dtype)
        dx, _ = tw.twell_rmsnorm_backward(to_dev(dy, dtype), to_dev(h, dtype), to_dev(w, dtype), eps)
        got = decode(from_dev(dx, dtype), dtype)
        assert np.isnan(got[1]).all() if eps == 0.0 else np.isfinite(got[1]).all()
        assert np.isfinite(got[others]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [300, 2048, 8200])
def test_infinities_beside_large_rows(dtype, d):
    v = _rows(d, [62, 0], 6, 53)
    v[2, d // 2] = np.inf
    v[3, d - 1] = np.nan
    h, w = to_storage(v, dtype), _weight(d, dtype, 54)
    y = decode(from_dev(tw.twell_rmsnorm(to_dev(h, dtype), to_dev(w, dtype), 1e-6).y, dtype), dtype)
    assert np.isnan(y[2, d // 2]) and not np.delete(y[2], d // 2).any() and np.isnan(y[3]).all()
    rest = [0, 1, 4, 5]
    y64 = rmsnorm(h, w, 1e-6, dtype)[rest]
    _close(y[rest], y64, 55 * U * np.abs(y64), dtype, "y")
