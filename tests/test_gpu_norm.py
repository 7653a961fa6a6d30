"""GPU parity of the residual RMS norm, its gradient and the row quantiser with
the float64 oracle.

Tolerances, from the arithmetic (u = 2^-24, storage rounding us = 2^-24 fp32,
2^-8 bf16):

* h and q are formed without sums and are compared bit for bit.
* A row's sum is a tree: at most 64 values per lane in sequence, 6 lane steps
  and at most 16 waves, so its relative error is below 90 u (all terms of the
  sum of squares are positive).  r = (mean + eps)^-1/2 halves it; the divide,
  the addition, the root and the two products of y add less than 10 u:
  |y - y64| <= 55 u |y64|, then one storage rounding.  scale: the same 55 u.
* dx: every term's products carry below 10 u, r and r^3 at most 165 u, the dot
  product 90 u of its absolute sum: 270 u (|dh| + r |g| + r^3 |h| mean|g h|)
  before the storage rounding.
* dweight: the terms carry 60 u, their sum runs over at most T / (workgroups)
  + 32 + 16 + 4 steps, below T + 60: (T + 120) u sum_t |dy h r|.
"""

import numpy as np
import pytest

from oracle.block import (norm_factor, quantize_rows, residual_sum, rmsnorm, rmsnorm_backward, rmsnorm_quantized)
from oracle.numerics import decode
from workloads.synth import to_storage

from gpu_util import assert_bitwise, from_dev, to_dev

pytestmark = pytest.mark.gpu

tw = pytest.importorskip("activation_sparse_transformer_bf16_amd")

U = 2.0 ** -24
US = {"f32": U, "bf16": 2.0 ** -8}
EPS = 1e-6

# rows, d: one element, below and above one 16-byte chunk, odd lengths, whole
# and partial chunks in each split of a row over lanes and waves
SHAPES = [(1, 1), (3, 7), (5, 64), (1, 2048), (67, 257), (130, 1000), (64, 512), (33, 2048), (9, 2049), (6, 4097),
          (5, 8192), (3, 16400), (2, 32768)]


def _data(T, d, dtype, seed):
    rng = np.random.default_rng(seed)
    channel = np.exp(0.5 * rng.standard_normal(d))
    channel[rng.integers(0, d, max(1, d // 256))] *= 12.0
    return to_storage(rng.standard_normal((T, d)) * channel * np.exp(0.3 * rng.standard_normal((T, 1))), dtype)


def _weight(d, dtype, seed):
    return to_storage(1.0 + 0.2 * np.random.default_rng(seed).standard_normal(d), dtype)


def _close(got, want, bound, dtype, what):
    err = np.abs(got - want)
    limit = bound + US[dtype] * (np.abs(want) + bound) + (2.0 ** -133 if dtype == "bf16" else 2.0 ** -149)
    bad = ~(err <= limit)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst {np.max(err / np.maximum(limit, 1e-300)):.3g} x the bound"


def _check_norm(out, x, res, w, dtype, quantized):
    h = residual_sum(x, res, dtype)
    if res is not None:
        assert_bitwise(from_dev(out.h.contiguous(), dtype), h, "h")
    if out.y is not None:
        y64 = rmsnorm(h, w, EPS, dtype)
        _close(decode(from_dev(out.y.contiguous(), dtype), dtype), y64, 55 * U * np.abs(y64), dtype, "y")
    if quantized:
        q, scale = rmsnorm_quantized(h, w, EPS, dtype)
        assert_bitwise(out.q.cpu().numpy(), q, "q")
        got = out.scale.cpu().numpy().astype(np.float64)
        assert np.all(np.abs(got - scale) <= 55 * U * scale)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,d", SHAPES)
def test_norm(dtype, T, d):
    print(f"norm {dtype} {T} x {d}", flush=True)
    x, res, w = _data(T, d, dtype, 1), _data(T, d, dtype, 2), _weight(d, dtype, 3)
    xd, rd, wd = to_dev(x, dtype), to_dev(res, dtype), to_dev(w, dtype)
    _check_norm(tw.twell_rmsnorm(xd, wd, EPS, rd, quantize=True), x, res, w, dtype, True)
    _check_norm(tw.twell_rmsnorm(xd, wd, EPS), x, None, w, dtype, False)
    only = tw.twell_rmsnorm(xd, wd, EPS, quantize=True, want_y=False)
    assert only.y is None and only.h is xd
    _check_norm(only, x, None, w, dtype, True)


def test_norm_longest_rows():
    for dtype, d in (("bf16", 65536), ("f32", 32768)):
        x, w = _data(2, d, dtype, 4), _weight(d, dtype, 5)
        _check_norm(tw.twell_rmsnorm(to_dev(x, dtype), to_dev(w, dtype), EPS, quantize=True), x, None, w, dtype, True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,d", SHAPES)
def test_quantize_rows(dtype, T, d):
    x = _data(T, d, dtype, 6)
    q, scale = tw.twell_quantize_rows(to_dev(x, dtype))
    want_q, want_s = quantize_rows(x, dtype)
    assert q.shape == (T, d) and (T == 1 or q.stride(0) % 16 == 0)
    assert_bitwise(q.cpu().numpy(), want_q, "q")
    assert np.all(np.abs(scale.cpu().numpy() - want_s) <= 2 * U * want_s)


def _bounds_backward(dy, h, w, dh, dtype):
    H, DY, W = decode(h, dtype), decode(dy, dtype), decode(w, dtype)
    r = norm_factor(h, EPS, dtype)[:, None]
    g = np.abs(DY * W)
    b = r * g + r ** 3 * np.abs(H) * np.mean(g * np.abs(H), axis=1, keepdims=True)
    if dh is not None:
        b = b + np.abs(decode(dh, dtype))
    return 270 * U * b, (H.shape[0] + 120) * U * np.sum(np.abs(DY * H) * r, axis=0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("stream", [False, True])
@pytest.mark.parametrize("T,d", SHAPES + [(2500, 96), (2051, 520)])
def test_norm_backward(dtype, stream, T, d):
    print(f"norm backward {dtype} {T} x {d} stream={stream}", flush=True)
    rng = np.random.default_rng(7)
    h, w = _data(T, d, dtype, 8), _weight(d, dtype, 9)
    dy = to_storage(rng.standard_normal((T, d)), dtype)
    dh = to_storage(rng.standard_normal((T, d)), dtype) if stream else None
    args = (to_dev(dy, dtype), to_dev(h, dtype), to_dev(w, dtype), EPS, to_dev(dh, dtype) if stream else None)
    dx, dw = tw.twell_rmsnorm_backward(*args)
    dx64, dw64 = rmsnorm_backward(dy, h, w, EPS, dtype, dh)
    bx, bw = _bounds_backward(dy, h, w, dh, dtype)
    _close(decode(from_dev(dx, dtype), dtype), dx64, bx, dtype, "dx")
    assert np.all(np.abs(dw.cpu().numpy() - dw64) <= bw)
    again = tw.twell_rmsnorm_backward(*args)
    assert_bitwise(from_dev(again[0], dtype), from_dev(dx, dtype), "dx of a second run")
    assert_bitwise(again[1].cpu().numpy(), dw.cpu().numpy(), "dweight of a second run")


def test_norm_backward_against_differences():
    # <dy, y(h, w)> in float64, central differences of step 1e-5: their own
    # error is below 1e-8 of the values here, the fp32 result's bound is above it
    T, d, step = 3, 37, 1e-5
    rng = np.random.default_rng(11)
    h, w = rng.standard_normal((T, d)).astype(np.float32), (1 + 0.2 * rng.standard_normal(d)).astype(np.float32)
    dy = rng.standard_normal((T, d)).astype(np.float32)
    dx, dw = tw.twell_rmsnorm_backward(to_dev(dy, "f32"), to_dev(h, "f32"), to_dev(w, "f32"), EPS)
    bx, bw = _bounds_backward(dy, h, w, None, "f32")

    def value(H, W):
        return np.sum(dy.astype(np.float64) * H / np.sqrt(np.mean(H * H, axis=1, keepdims=True) + EPS) * W)

    H, W = h.astype(np.float64), w.astype(np.float64)
    for j in range(d):
        e = np.zeros(d)
        e[j] = step
        assert abs((value(H, W + e) - value(H, W - e)) / (2 * step) - float(dw[j])) <= bw[j] + 1e-7
        for t in range(T):
            E = np.zeros((T, d))
            E[t, j] = step
            assert abs((value(H + E, W) - value(H - E, W)) / (2 * step) - float(dx[t, j])) <= bx[t, j] + 1e-7


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,ld,off", [(100, 128, 0), (100, 101, 1), (520, 1040, 8), (77, 333, 3), (2048, 2050, 1)])
def test_row_strides_and_alignment(dtype, d, ld, off):
    # rows inside wider buffers, at offsets that break the 16-byte alignment;
    # what lies around the outputs stays as it was
    import torch
    T = 13
    x, res, w = _data(T, d, dtype, 12), _data(T, d, dtype, 13), _weight(d, dtype, 14)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16

    def wide(a=None):
        buf = torch.full((T, ld + 16), 7.0, dtype=dt, device="cuda:0")
        view = buf[:, off:off + d]
        if a is not None:
            view.copy_(to_dev(a, dtype))
        return buf, view

    (_, xd), (_, rd), (hb, hd), (yb, yd) = wide(x), wide(res), wide(), wide()
    qb = torch.full((T, (d + 15) // 16 * 16 + 32), 55, dtype=torch.int8, device="cuda:0")
    q, scale = qb[:, 16:16 + d], torch.empty(T, device="cuda:0")
    out = tw.twell_rmsnorm(xd, to_dev(w, dtype), EPS, rd, h=hd, y=yd, q=q, scale=scale)
    _check_norm(out, x, res, w, dtype, True)
    for buf in (hb, yb):
        assert bool((buf[:, :off] == 7).all()) and bool((buf[:, off + d:] == 7).all())
    assert bool((qb[:, :16] == 55).all()) and bool((qb[:, 16 + d:] == 55).all())
    # the gradient on the same kinds of views, and the quantiser
    dy, dh = _data(T, d, dtype, 15), _data(T, d, dtype, 16)
    (_, dyd), (_, dhd), (gb, gd) = wide(dy), wide(dh), wide()
    dx, dw = tw.twell_rmsnorm_backward(dyd, xd, to_dev(w, dtype), EPS, dh=dhd, dx=gd)
    dx64, dw64 = rmsnorm_backward(dy, x, w, EPS, dtype, dh)
    bx, bw = _bounds_backward(dy, x, w, dh, dtype)
    _close(decode(from_dev(gd.contiguous(), dtype), dtype), dx64, bx, dtype, "dx")
    assert np.all(np.abs(dw.cpu().numpy() - dw64) <= bw)
    assert bool((gb[:, :off] == 7).all()) and bool((gb[:, off + d:] == 7).all())
    q2, s2 = tw.twell_quantize_rows(xd)
    assert_bitwise(q2.cpu().numpy(), quantize_rows(x, dtype)[0], "q of strided rows")


LENGTHS = [3, 4, 5, 8, 9, 15, 255, 257, 511, 513, 1023, 1025, 2047, 2049, 4095, 4097, 8191, 8193, 16383, 16385, 32767]


@pytest.mark.parametrize("dtype,d", [(t, d) for t in ("f32", "bf16") for d in LENGTHS] + [("bf16", 65535)])
def test_unaligned_rows_of_every_length(dtype, d):
    # rows one element apart in a buffer of NaN, so at every alignment, ending
    # before, at and behind each edge of a lane's, a wave's and a workgroup's
    # part: nothing around a row may reach its results or change.  The outputs
    # lie over inputs.
    import torch
    T = 5
    x, res, w = _data(T, d, dtype, 31), _data(T, d, dtype, 32), _weight(d, dtype, 33)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16

    def apart(a):
        buf = torch.full((T * (d + 1) + 1,), float("nan"), dtype=dt, device="cuda:0")
        view = buf[1:].view(T, d + 1)[:, :d]
        view.copy_(to_dev(a, dtype))
        return buf, view

    wd = apart(np.repeat(w[None], T, 0))[1][1]
    q, scale = tw.twell_quantize_rows(apart(x)[1])
    assert_bitwise(q.cpu().numpy(), quantize_rows(x, dtype)[0], "q of the quantiser")
    (xb, xd), (rb, rd) = apart(x), apart(res)
    out = tw.twell_rmsnorm(xd, wd, EPS, rd, quantize=True, h=rd, y=xd)
    _check_norm(out, x, res, w, dtype, True)
    dy, dh = _data(T, d, dtype, 34), _data(T, d, dtype, 35)
    h = residual_sum(x, res, dtype)
    dx64, dw64 = rmsnorm_backward(dy, h, w, EPS, dtype, dh)
    bx, bw = _bounds_backward(dy, h, w, dh, dtype)
    for over in ("dh", "dy"):
        (yb, yd), (gb, gd) = apart(dy), apart(dh)
        dx, dw = tw.twell_rmsnorm_backward(yd, rd, wd, EPS, dh=gd, dx=gd if over == "dh" else yd)
        _close(decode(from_dev(dx.contiguous(), dtype), dtype), dx64, bx, dtype, f"dx over {over}")
        assert np.all(np.abs(dw.cpu().numpy() - dw64) <= bw)
        for buf in (xb, rb, yb, gb):
            assert bool(buf[::d + 1].isnan().all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [200, 4100])
def test_outputs_over_inputs(dtype, d):
    T = 21
    x, res, w = _data(T, d, dtype, 17), _data(T, d, dtype, 18), _weight(d, dtype, 19)
    wd = to_dev(w, dtype)
    want = tw.twell_rmsnorm(to_dev(x, dtype), wd, EPS, to_dev(res, dtype))
    xd, rd = to_dev(x, dtype), to_dev(res, dtype)
    out = tw.twell_rmsnorm(xd, wd, EPS, rd, h=rd, y=xd)  # the stream updated in place
    assert out.h is rd and out.y is xd
    assert_bitwise(from_dev(rd, dtype), from_dev(want.h, dtype), "h in place")
    assert_bitwise(from_dev(xd, dtype), from_dev(want.y, dtype), "y in place")
    dy, dh = to_dev(_data(T, d, dtype, 20), dtype), to_dev(_data(T, d, dtype, 21), dtype)
    ref, _ = tw.twell_rmsnorm_backward(dy, rd, wd, EPS, dh=dh)
    got, _ = tw.twell_rmsnorm_backward(dy, rd, wd, EPS, dh=dh, dx=dh)
    assert got is dh
    assert_bitwise(from_dev(got, dtype), from_dev(ref, dtype), "dx over dh")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_special_rows(dtype):
    # zeros, values far below 2^-100, one infinity, one NaN, an ordinary row
    d = 300
    v = np.random.default_rng(22).standard_normal((5, d))
    v[0] = 0.0
    v[1] *= 2.0 ** -120
    v[2, 17] = np.inf
    v[3, 299] = np.nan
    x = to_storage(v, dtype)
    w = _weight(d, dtype, 23)
    out = tw.twell_rmsnorm(to_dev(x, dtype), to_dev(w, dtype), EPS, quantize=True)
    y = decode(from_dev(out.y, dtype), dtype)
    q, scale = out.q.cpu().numpy(), out.scale.cpu().numpy()
    want_q, want_s = rmsnorm_quantized(x, w, EPS, dtype)
    assert not y[0].any()
    assert np.isnan(y[2, 17]) and not np.delete(y[2], 17).any()      # r = 0 for an infinite mean square
    assert np.isnan(y[3]).all()
    for t in (0, 1, 4):
        assert_bitwise(q[t], want_q[t], f"q of row {t}")
        assert abs(scale[t] - want_s[t]) <= 55 * U * want_s[t]
    for t in (2, 3):
        assert not q[t].any() and np.isnan(scale[t])
    q2, s2 = tw.twell_quantize_rows(to_dev(x, dtype))
    assert_bitwise(q2.cpu().numpy(), quantize_rows(x, dtype)[0], "q")
    assert np.array_equal(np.isnan(s2.cpu().numpy()), [False, False, True, True, False])
    dy = _data(5, d, dtype, 24)
    dx, _ = tw.twell_rmsnorm_backward(to_dev(dy, dtype), to_dev(x, dtype), to_dev(w, dtype), EPS)
    dx64, _ = rmsnorm_backward(dy, x, w, EPS, dtype)
    bx, _ = _bounds_backward(dy, x, w, None, dtype)
    for t in (0, 1, 4):
        _close(decode(from_dev(dx, dtype), dtype)[t], dx64[t], bx[t], dtype, f"dx of row {t}")


def test_no_rows():
    import torch
    for dtype in (torch.float32, torch.bfloat16):
        x = torch.empty((0, 96), dtype=dtype, device="cuda:0")
        w = torch.ones(96, dtype=dtype, device="cuda:0")
        out = tw.twell_rmsnorm(x, w, EPS, quantize=True)
        assert out.y.shape == (0, 96) and out.q.shape == (0, 96) and out.scale.shape == (0,)
        dx, dw = tw.twell_rmsnorm_backward(x, x, w, EPS)
        assert dx.shape == (0, 96) and not dw.any()


def test_more_rows_than_workgroups():
    # over 2^22 rows: each workgroup takes several row groups
    import torch
    T, d = 4 * (1 << 20) + 77, 8
    g = torch.Generator(device="cuda:0")
    g.manual_seed(25)
    x = torch.randn(T, d, generator=g, device="cuda:0")
    w = torch.ones(d, device="cuda:0")
    out = tw.twell_rmsnorm(x, w, EPS, quantize=True)
    rows = np.r_[0:5, (1 << 22) - 3:(1 << 22) + 3, T - 5:T]
    xs = x[torch.from_numpy(rows).cuda()].cpu().numpy()
    ys = out.y[torch.from_numpy(rows).cuda()].cpu().numpy()
    y64 = rmsnorm(xs, np.ones(d, np.float32), EPS, "f32")
    _close(ys.astype(np.float64), y64, 55 * U * np.abs(y64), "f32", "y")
    assert_bitwise(out.q[torch.from_numpy(rows).cuda()].cpu().numpy(),
                   rmsnorm_quantized(xs, np.ones(d, np.float32), EPS, "f32")[0], "q")
    assert bool((out.y != 0).any(1).all())


def test_rows_beyond_32_bit_offsets():
    # three rows, each 2^31 elements after the one before
    import torch
    d, ld = 192, (1 << 31) + 64
    x, w = _data(3, d, "bf16", 26), _weight(d, "bf16", 27)
    buf = torch.empty(2 * ld + 256, dtype=torch.bfloat16, device="cuda:0")
    xd = buf.as_strided((3, d), (ld, 1))
    xd.copy_(to_dev(x, "bf16"))
    _check_norm(tw.twell_rmsnorm(xd, to_dev(w, "bf16"), EPS, quantize=True), x, None, w, "bf16", True)


def test_on_another_stream():
    import torch
    T, d = 512, 1024
    x, w = _data(T, d, "bf16", 28), _weight(d, "bf16", 29)
    xd, wd = to_dev(x, "bf16"), to_dev(w, "bf16")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = tw.twell_rmsnorm(xd, wd, EPS, quantize=True)
        dx, dw = tw.twell_rmsnorm_backward(xd, xd, wd, EPS)
    s.synchronize()
    _check_norm(out, x, None, w, "bf16", True)
    dx64, dw64 = rmsnorm_backward(x, x, w, EPS, "bf16")
    bx, bw = _bounds_backward(x, x, w, None, "bf16")
    _close(decode(from_dev(dx, "bf16"), "bf16"), dx64, bx, "bf16", "dx")
    assert np.all(np.abs(dw.cpu().numpy() - dw64) <= bw)


def test_refusals():
    import torch
    x = torch.zeros(4, 64, device="cuda:0")
    w = torch.ones(64, device="cuda:0")
    with pytest.raises(TypeError):
        tw.twell_rmsnorm(x, w.bfloat16())
    with pytest.raises(ValueError):
        tw.twell_rmsnorm(x, w[:63])
    with pytest.raises(ValueError):
        tw.twell_rmsnorm(x.t(), w[:4])                       # rows without unit stride
    with pytest.raises(ValueError):
        tw.twell_rmsnorm(x, w, residual=x[:3])
    with pytest.raises(ValueError):
        tw.twell_rmsnorm(x, w, q=torch.zeros(4, 64, dtype=torch.int8, device="cuda:0"))   # no scale
    with pytest.raises(tw.TwellError):
        tw.twell_rmsnorm(x, w, eps=-1.0)
    with pytest.raises(tw.TwellError):
        tw.twell_rmsnorm(x[:1].expand(4, 64), w)             # rows on top of each other
    with pytest.raises(ValueError):
        tw.twell_rmsnorm(x, w, q=torch.zeros(4, 72, dtype=torch.int8, device="cuda:0")[:, :64],
                         scale=torch.zeros(4, device="cuda:0"))  # stride not a multiple of 16
    with pytest.raises(ValueError):
        tw.twell_rmsnorm_backward(x, x, w, dh=x[:2])
    with pytest.raises(TypeError):
        tw.twell_rmsnorm_backward(x, x, w, dweight=torch.zeros(64, dtype=torch.bfloat16, device="cuda:0"))
