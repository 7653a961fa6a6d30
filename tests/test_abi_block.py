"""The block operators reject bad arguments before any HIP call (CPU only: no
kernel is ever launched here)."""

import ctypes

import pytest

twell = pytest.importorskip("activation_sparse_transformer_bf16_amd")

FAKE = 0x100000  # a non-null, 256-byte aligned address that must never be dereferenced
L = twell.lib()
INVALID, UNSUPPORTED, WORKSPACE = twell.TWELL_ERR_INVALID_ARG, twell.TWELL_ERR_UNSUPPORTED, twell.TWELL_ERR_WORKSPACE
F32, BF16 = twell.TWELL_F32, twell.TWELL_BF16


def _q(rows=8, cols=512, ld=512, q=FAKE, scale=FAKE):
    return twell.TwellInt8C(rows, cols, ld, q, scale)


def _ref(q):
    return None if q is None else ctypes.byref(q)


def norm(x=FAKE, ld_x=512, residual=None, ld_r=512, weight=FAKE, eps=1e-6, rows=8, d=512, dtype=BF16, h=None, ld_h=512,
         y=FAKE, ld_y=512, q=None):
    return L.twell_rmsnorm(x, ld_x, residual, ld_r, weight, eps, rows, d, dtype, h, ld_h, y, ld_y, _ref(q), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=7), INVALID),
    (dict(rows=-1), INVALID),
    (dict(d=0), INVALID),
    (dict(d=65537, ld_x=70000), UNSUPPORTED),
    (dict(d=32769, ld_x=70000, dtype=F32), UNSUPPORTED),
    (dict(x=None), INVALID),
    (dict(x=FAKE + 1), UNSUPPORTED),
    (dict(x=FAKE + 2, dtype=F32), UNSUPPORTED),
    (dict(ld_x=511), INVALID),
    (dict(ld_x=-512), INVALID),
    (dict(ld_x=1 << 50), INVALID),
    (dict(residual=FAKE, ld_r=100), INVALID),
    (dict(h=FAKE, ld_h=100), INVALID),
    (dict(y=FAKE, ld_y=100), INVALID),
    (dict(weight=None), INVALID),
    (dict(weight=FAKE + 1), UNSUPPORTED),
    (dict(y=None), INVALID),                               # no output at all
    (dict(eps=-1e-6), INVALID),
    (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID),
    (dict(q=_q(rows=7)), INVALID),
    (dict(q=_q(cols=511)), INVALID),
    (dict(q=_q(ld=520)), UNSUPPORTED),                     # stride not a multiple of 16
    (dict(q=_q(ld=496)), INVALID),                         # below the row length
    (dict(q=_q(q=FAKE + 8)), UNSUPPORTED),
    (dict(q=_q(q=None)), INVALID),
    (dict(q=_q(scale=None)), INVALID),
    (dict(q=_q(scale=FAKE + 2)), UNSUPPORTED),
])
def test_norm_validation(kw, status):
    assert norm(**kw) == status
    assert twell.twell_last_error() != ""


def test_norm_of_no_rows_launches_nothing():
    assert norm(rows=0, x=None, y=None, weight=None) == twell.TWELL_OK
    assert norm(rows=0, x=None, y=None, weight=None, q=_q(rows=0, q=None, scale=None)) == twell.TWELL_OK


def back(dy=FAKE, ld_dy=512, h=FAKE, ld_h=512, weight=FAKE, dh=None, ld_dh=512, eps=1e-6, rows=8, d=512, dtype=BF16,
         dx=FAKE, ld_dx=512, dweight=FAKE, ws=FAKE, ws_bytes=1 << 40):
    return L.twell_rmsnorm_backward(dy, ld_dy, h, ld_h, weight, dh, ld_dh, eps, rows, d, dtype, dx, ld_dx, dweight,
                                    ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=-1), INVALID), (dict(rows=-3), INVALID), (dict(d=-1), INVALID), (dict(d=70000, ld_dy=70000), UNSUPPORTED),
    (dict(dy=None), INVALID), (dict(h=None), INVALID), (dict(dx=None), INVALID), (dict(weight=None), INVALID),
    (dict(dweight=None), INVALID), (dict(dweight=FAKE + 2), UNSUPPORTED), (dict(dy=FAKE + 1), UNSUPPORTED),
    (dict(ld_dy=5), INVALID), (dict(ld_h=5), INVALID), (dict(ld_dx=5), INVALID), (dict(dh=FAKE, ld_dh=5), INVALID),
    (dict(eps=-1.0), INVALID), (dict(ws=None), WORKSPACE), (dict(ws_bytes=100), WORKSPACE),
    (dict(ws=FAKE + 16), UNSUPPORTED),
])
def test_norm_backward_validation(kw, status):
    assert back(**kw) == status
    assert twell.twell_last_error() != ""


def test_norm_backward_workspace():
    import torch
    ws = twell.twell_rmsnorm_backward_workspace_size
    # one fp32 row of d values for each workgroup, at most 256 of them
    assert ws(8192, 2048, torch.bfloat16) == 256 * 2048 * 4
    assert ws(1, 2048, torch.bfloat16) == 2048 * 4
    assert ws(0, 7, torch.float32) == 256
    assert ws(-1, 64, torch.float32) == 0 and ws(4, 40000, torch.float32) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INVALID), (dict(ld_x=511), INVALID), (dict(dtype=9), INVALID), (dict(x=FAKE + 1), UNSUPPORTED),
    (dict(out=None), INVALID), (dict(out=_q(rows=-1)), INVALID), (dict(out=_q(cols=0)), INVALID),
    (dict(out=_q(ld=516)), UNSUPPORTED), (dict(out=_q(cols=70000, ld=70016), ld_x=70000), UNSUPPORTED),
])
def test_quantize_validation(kw, status):
    a = dict(x=FAKE, ld_x=512, dtype=BF16, out=_q())
    a.update(kw)
    assert L.twell_quantize_rows(a["x"], a["ld_x"], a["dtype"], _ref(a["out"]), None) == status
    assert twell.twell_last_error() != ""


@pytest.mark.parametrize("kw,status", [
    (dict(a=None), INVALID), (dict(b=None), INVALID), (dict(dtype=2), INVALID), (dict(y=None), INVALID),
    (dict(b=_q(cols=500)), INVALID),                                         # different row lengths
    (dict(a=_q(cols=65537, ld=65552), b=_q(cols=65537, ld=65552)), UNSUPPORTED),
    (dict(a=_q(ld=500)), INVALID), (dict(a=_q(ld=514)), UNSUPPORTED), (dict(b=_q(q=FAKE + 4)), UNSUPPORTED),
    (dict(a=_q(scale=None)), INVALID), (dict(ld_y=7), INVALID), (dict(y=FAKE + 1), UNSUPPORTED),
    (dict(a=_q(rows=(1 << 26) + 1)), UNSUPPORTED), (dict(b=_q(rows=(1 << 26) + 1), ld_y=1 << 27), UNSUPPORTED),
    (dict(bias=FAKE + 1), UNSUPPORTED), (dict(ws=FAKE + 16), UNSUPPORTED),
    (dict(a=_q(rows=64, cols=40000, ld=40000), b=_q(cols=40000, ld=40000), ws=None), WORKSPACE),
    (dict(a=_q(rows=64, cols=40000, ld=40000), b=_q(cols=40000, ld=40000), ws_bytes=100), WORKSPACE),
])
def test_product_validation(kw, status):
    a = dict(a=_q(), b=_q(), bias=None, dtype=BF16, y=FAKE, ld_y=8, ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    assert L.twell_int8_matmul(_ref(a["a"]), _ref(a["b"]), a["bias"], a["dtype"], a["y"], a["ld_y"], a["ws"],
                               a["ws_bytes"], None) == status
    assert twell.twell_last_error() != ""


def test_product_workspace():
    ws = twell.twell_int8_matmul_workspace_size
    assert ws(1, 8192, 2048) == 0 and ws(64, 2048, 8192) == 0 and ws(8192, 8192, 2048) == 0 and ws(0, 64, 64) == 0
    assert ws(64, 64, 0) == 0 and ws(64, 64, 70000) == 0 and ws(-1, 64, 64) == 0
    # few tiles and a long K: whole [M][N] matrices of 4-byte sums
    for M, N, K in [(40, 515, 40000), (17, 333, 65536), (300, 260, 20000), (2349, 39, 29705)]:
        n = ws(M, N, K)
        assert n > 0 and n % (M * ((N + 3) // 4 * 4) * 4) == 0 and n <= 64 << 20, (M, N, K, n)


def test_empty_products_launch_nothing():
    none = _q(rows=0, q=None, scale=None)
    assert L.twell_int8_matmul(_ref(none), _ref(_q()), None, BF16, None, 8, None, 0, None) == twell.TWELL_OK
    assert L.twell_int8_matmul(_ref(_q()), _ref(none), None, BF16, None, 0, None, 0, None) == twell.TWELL_OK
    assert L.twell_quantize_rows(None, 512, BF16, _ref(none), None) == twell.TWELL_OK


def test_binding_refuses_tensors_that_are_not_on_the_gpu():
    import torch
    x, w = torch.zeros(4, 64), torch.ones(64)
    with pytest.raises(ValueError):
        twell.twell_rmsnorm(x, w)
    with pytest.raises(ValueError):
        twell.twell_rmsnorm_backward(x, x, w)
    with pytest.raises(ValueError):
        twell.twell_quantize_rows(x)
    q, s = torch.zeros(4, 64, dtype=torch.int8), torch.ones(4)
    with pytest.raises(ValueError):
        twell.twell_int8_matmul(q, s, q, s)
    with pytest.raises(TypeError):
        twell.twell_quantize_rows(x.half())
    with pytest.raises(ValueError):
        twell.twell_quantize_rows(torch.zeros(64))
