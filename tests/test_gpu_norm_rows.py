"""The norm's gradient over several groups of rows per workgroup, for each split
of a row over waves and lanes, in both types, with whole, unaligned and tiny
rows, and with its result over its inputs.

References are float64 on the GPU, from the formulas.  Tolerances (u = 2^-24): dx
within 270 u of its absolute terms and one storage rounding, as test_gpu_norm.py
derives it.  dweight: a wave adds at most n = rows / (256 groups) + 1 rows, a
workgroup its at most 16 row groups, then 8 partial rows a thread and 32 threads;
the terms carry r's 51 u and three roundings: (n + 120) u sum_t |dy h r|.
"""

import pytest

from gpu_util import torch_dtype

pytestmark = pytest.mark.gpu

tw = pytest.importorskip("activation_sparse_transformer_bf16_amd")

U = 2.0 ** -24
US = {"f32": U, "bf16": 2.0 ** -8}
EPS = 1e-6
WORKGROUPS, WAVES = 256, 16

# Waves a row -> row length in bf16 (fp32: half of it): 1, 2, 4, 8, 16, 32, 64 and
# 128 chunks of 64 x 16 bytes at most, in the last two four and eight chunks a lane.
SPLITS = {"1a": (1, 256), "1b": (1, 1000), "2": (2, 2000), "4": (4, 4000), "8": (8, 8000), "16a": (16, 12000),
          "16b": (16, 20000), "16c": (16, 40000), "tiny": (1, 6)}


def _case(split, dtype, odd):
    waves, d = SPLITS[split]
    d = (d if dtype == "bf16" else d // 2) + odd
    # more than two whole rounds of the workgroups' row groups, the last one ragged
    return WAVES // waves, 2 * WORKGROUPS * (WAVES // waves) + 5 * WAVES + 3, d


def _inputs(T, d, dtype, seed):
    import torch
    g = torch.Generator(device="cuda:0")
    g.manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda:0")  # noqa: E731
    dt = torch_dtype(dtype)
    return (rand(T, d).to(dt), (rand(T, d) * torch.exp(0.5 * rand(T, 1))).to(dt), (1 + 0.2 * rand(d)).to(dt),
            rand(T, d).to(dt))


def _check(dx, dw, dy, h, w, dh, dtype, n):
    H, DY = h.double(), dy.double()
    r = 1.0 / (H.pow(2).mean(1, keepdim=True) + EPS).sqrt()
    g = DY * w.double()
    want = r * g - r ** 3 * H * (g * H).mean(1, keepdim=True)
    bound = r * g.abs() + r ** 3 * H.abs() * (g * H).abs().mean(1, keepdim=True)
    if dh is not None:
        want, bound = want + dh.double(), bound + dh.double().abs()
    bound = 270 * U * bound
    limit = bound + US[dtype] * (want.abs() + bound) + 2.0 ** -133
    bad = ~((dx.double() - want).abs() <= limit)
    assert not bool(bad.any()), f"dx: {int(bad.sum())} of {bad.numel()} outside, first at {bad.nonzero()[0].tolist()}"
    terms = DY * H * r
    bad = ~((dw.double() - terms.sum(0)).abs() <= (n + 120) * U * terms.abs().sum(0))
    assert not bool(bad.any()), f"dweight: {int(bad.sum())} of {bad.numel()} outside"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("odd", [0, 1])
@pytest.mark.parametrize("split", SPLITS)
def test_gradient_over_several_row_groups(dtype, odd, split):
    import torch
    groups, T, d = _case(split, dtype, odd)
    print(f"gradient {dtype} {T} x {d}", flush=True)
    n = T // (WORKGROUPS * groups) + 1
    dy, h, w, dh = _inputs(T, d, dtype, 61)
    dx, dw = tw.twell_rmsnorm_backward(dy, h, w, EPS, dh=dh)
    _check(dx, dw, dy, h, w, dh, dtype, n)
    again = tw.twell_rmsnorm_backward(dy, h, w, EPS, dh=dh)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
    alone, dw2 = tw.twell_rmsnorm_backward(dy, h, w, EPS)
    _check(alone, dw2, dy, h, w, None, dtype, n)
    assert torch.equal(dw2, dw)
    # the result over either input
    over = dh.clone()
    assert tw.twell_rmsnorm_backward(dy, h, w, EPS, dh=over, dx=over)[0] is over and torch.equal(over, dx)
    over = dy.clone()
    got, dw3 = tw.twell_rmsnorm_backward(over, h, w, EPS, dh=dh, dx=over)
    assert torch.equal(got, dx) and torch.equal(dw3, dw)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("split", ["1b", "2", "8", "16b", "16c"])
def test_gradient_of_strided_row_groups(dtype, split):
    # rows at odd distances inside wider buffers, whose other bytes stay
    import torch
    groups, T, d = _case(split, dtype, 1)
    print(f"gradient {dtype} {T} x {d}, strided", flush=True)
    dy, h, w, dh = _inputs(T, d, dtype, 62)

    def wide(t):
        buf = torch.full((T, d + 4), 7.0, dtype=t.dtype, device="cuda:0")
        buf[:, 3:3 + d] = t
        return buf, buf[:, 3:3 + d]

    (_, dyv), (_, hv), (_, dhv), (ob, ov) = wide(dy), wide(h), wide(dh), wide(dy)
    _, dw = tw.twell_rmsnorm_backward(dyv, hv, w, EPS, dh=dhv, dx=ov)
    _check(ov, dw, dy, h, w, dh, dtype, T // (WORKGROUPS * groups) + 1)
    assert bool((ob[:, :3] == 7).all()) and bool((ob[:, 3 + d:] == 7).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("odd", [0, 1])
@pytest.mark.parametrize("split", SPLITS)
def test_norm_and_quantiser_of_many_rows(dtype, odd, split):
    # h = x + residual bit for bit, y within 55 u and one rounding, 8-bit values
    # within half a step of z; the norm's result over its inputs
    import torch
    _, T, d = _case(split, dtype, odd)
    print(f"norm {dtype} {T} x {d}", flush=True)
    x, res, w, _ = _inputs(T, d, dtype, 63)
    out = tw.twell_rmsnorm(x, w, EPS, residual=res, quantize=True)
    h = (x.float() + res.float()).to(x.dtype)
    assert torch.equal(out.h, h)
    H, W = h.double(), w.double()
    r = 1.0 / (H.pow(2).mean(1, keepdim=True) + EPS).sqrt()
    want = H * r * W
    bound = 55 * U * want.abs()
    assert bool(((out.y.double() - want).abs() <= bound + US[dtype] * (want.abs() + bound) + 2.0 ** -133).all())
    top = (h.float() * w.float()).abs().amax(1).clamp_min(2.0 ** -100).double()
    scale = r[:, 0] * top / 127
    assert bool(((out.scale.double() - scale).abs() <= 55 * U * scale).all())
    step = top[:, None] / 127
    assert bool(((out.q.double() * step - H * W).abs() <= 0.5 * step * (1 + 2.0 ** -14)).all())
    xd, rd = x.clone(), res.clone()
    tw.twell_rmsnorm(xd, w, EPS, residual=rd, h=rd, y=xd)
    assert torch.equal(rd, out.h) and torch.equal(xd, out.y)
