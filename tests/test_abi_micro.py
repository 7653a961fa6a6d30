"""The microscaled operators and the optimiser reject bad arguments before any HIP
call (CPU only: no kernel is ever launched here)."""

import ctypes

import pytest

tw = pytest.importorskip("activation_sparse_transformer_bf16_amd")

FAKE = 0x100000  # a non-null, 256-byte aligned address that must never be dereferenced
L = tw.lib()
OK, INVALID, UNSUPPORTED, WORKSPACE = (tw.TWELL_OK, tw.TWELL_ERR_INVALID_ARG, tw.TWELL_ERR_UNSUPPORTED,
                                       tw.TWELL_ERR_WORKSPACE)
F32, BF16 = tw.TWELL_F32, tw.TWELL_BF16
BIG = 1 << 40


def _q(rows=8, cols=512, ld=256, q=FAKE, ld_scale=16, scale=FAKE, factor=None):
    return tw.TwellMx4C(rows, cols, ld, q, ld_scale, scale, factor)


def _ref(q):
    return None if q is None else ctypes.byref(q)


BAD_ROWS = [
    (dict(rows=-1), INVALID),
    (dict(cols=0), INVALID),
    (dict(ld=240), INVALID),                # below the row length
    (dict(cols=513, ld=256), INVALID),      # 257 bytes
    (dict(ld=264), UNSUPPORTED),            # not a multiple of 16
    (dict(ld=1 << 50), INVALID),
    (dict(cols=(1 << 30) + 1, ld=1 << 30, ld_scale=1 << 26), UNSUPPORTED),
    (dict(q=None), INVALID),
    (dict(q=FAKE + 8), UNSUPPORTED),
    (dict(ld_scale=0), INVALID),
    (dict(cols=544, ld=272, ld_scale=16), INVALID),  # 17 blocks
    (dict(ld_scale=24), UNSUPPORTED),
    (dict(ld_scale=-16), INVALID),
    (dict(scale=None), INVALID),
    (dict(scale=FAKE + 4), UNSUPPORTED),
    (dict(factor=FAKE + 2), UNSUPPORTED),
]


def quantize(x=FAKE, ld_x=1024, dtype=BF16, out=_q()):
    return L.twell_quantize_mx4(x, ld_x, dtype, _ref(out), None)


def dequantize(q=_q(), dtype=BF16, y=FAKE, ld_y=1024):
    return L.twell_dequantize_mx4(_ref(q), dtype, y, ld_y, None)


def norm(x=FAKE, ld_x=512, residual=None, ld_r=512, weight=FAKE, eps=1e-6, rows=8, d=512, dtype=BF16, h=None, ld_h=512,
         y=FAKE, ld_y=512, q=_q(factor=FAKE)):
    return L.twell_rmsnorm_mx4(x, ld_x, residual, ld_r, weight, eps, rows, d, dtype, h, ld_h, y, ld_y, _ref(q), None)


def product(a=_q(), b=_q(rows=16), bias=None, dtype=BF16, y=FAKE, ld_y=16, ws=FAKE, n=BIG):
    return L.twell_mx4_matmul(_ref(a), _ref(b), bias, dtype, y, ld_y, ws, n, None)


@pytest.mark.parametrize("kw,status", BAD_ROWS)
def test_rows_validation(kw, status):
    assert dequantize(q=_q(**kw)) == status
    assert tw.twell_last_error() != ""
    assert product(a=_q(**kw)) == status and product(b=_q(**kw)) == status
    if "factor" not in kw:
        assert quantize(out=_q(**kw)) == status
    if "rows" not in kw and "cols" not in kw:  # the norm's own sizes come first
        assert norm(q=_q(**{"factor": FAKE, **kw})) == status


@pytest.mark.parametrize("call,kw,status", [
    (quantize, dict(out=None), INVALID),
    (quantize, dict(x=None), INVALID),
    (quantize, dict(x=FAKE + 1), UNSUPPORTED),
    (quantize, dict(x=FAKE + 2, dtype=F32), UNSUPPORTED),
    (quantize, dict(ld_x=511), INVALID),
    (quantize, dict(dtype=5), INVALID),
    (quantize, dict(out=_q(factor=FAKE)), INVALID),
    (dequantize, dict(q=None), INVALID),
    (dequantize, dict(y=None), INVALID),
    (dequantize, dict(y=FAKE + 2, dtype=F32), UNSUPPORTED),
    (dequantize, dict(ld_y=500), INVALID),
    (dequantize, dict(dtype=-1), INVALID),
    (norm, dict(dtype=7), INVALID),
    (norm, dict(rows=-1), INVALID),
    (norm, dict(d=65537, ld_x=70000), UNSUPPORTED),
    (norm, dict(x=None), INVALID),
    (norm, dict(ld_x=511), INVALID),
    (norm, dict(residual=FAKE, ld_r=100), INVALID),
    (norm, dict(h=FAKE, ld_h=100), INVALID),
    (norm, dict(y=FAKE + 1), UNSUPPORTED),
    (norm, dict(weight=None), INVALID),
    (norm, dict(weight=FAKE + 1), UNSUPPORTED),
    (norm, dict(eps=-1.0), INVALID),
    (norm, dict(q=None), INVALID),
    (norm, dict(q=_q()), INVALID),                                  # no factor
    (norm, dict(q=_q(rows=7, factor=FAKE)), INVALID),
    (norm, dict(q=_q(cols=480, factor=FAKE)), INVALID),
    (product, dict(a=None), INVALID),
    (product, dict(b=None), INVALID),
    (product, dict(a=_q(cols=480)), INVALID),                       # different columns
    (product, dict(a=_q(cols=(1 << 20) + 32, ld=1 << 20, ld_scale=1 << 16),
                   b=_q(cols=(1 << 20) + 32, ld=1 << 20, ld_scale=1 << 16)), UNSUPPORTED),
    (product, dict(a=_q(rows=(1 << 26) + 1)), UNSUPPORTED),
    (product, dict(y=None), INVALID),
    (product, dict(ld_y=15), INVALID),
    (product, dict(y=FAKE + 1), UNSUPPORTED),
    (product, dict(bias=FAKE + 2), UNSUPPORTED),
    (product, dict(dtype=9), INVALID),
])
def test_validation(call, kw, status):
    assert call(**kw) == status
    assert tw.twell_last_error() != ""


def test_no_rows_launch_nothing():
    none = _q(rows=0, q=None, scale=None)
    assert quantize(x=None, out=none) == OK and dequantize(q=none, y=None) == OK
    assert norm(x=None, rows=0, y=None, weight=None, q=none) == OK
    assert product(a=none, y=None) == OK and product(b=none, y=None) == OK


def test_binding_refuses_rows_beyond_32_bits():
    # (ctypes would pass their low 32 bits)
    torch = pytest.importorskip("torch")
    big = tw.Mx4Rows.empty((1 << 31) + 3, 32, "meta")
    small = tw.Mx4Rows.empty(3, 32, "meta")
    for call in (lambda: tw.twell_dequantize_mx4(big), lambda: tw.twell_mx4_matmul(big, small),
                 lambda: tw.twell_mx4_matmul(small, big),
                 lambda: tw.twell_quantize_mx4(torch.empty((1 << 31) + 3, 32, dtype=torch.bfloat16, device="meta"))):
        with pytest.raises(ValueError, match="2147483651|meta"):
            call()


def test_product_workspace():
    size = tw.twell_mx4_matmul_workspace_size
    for M, N, K in [(0, 5, 5), (5, 0, 5), (5, 5, 0), (-1, 5, 5), (5, 5, (1 << 20) + 1), ((1 << 26) + 1, 1, 32),
                    (1 << 40, 5, 5)]:
        assert size(M, N, K) == 0
    # some product is cut into ranges of K, and refuses less
    M, N, K = next((m, n, k) for m in (512, 1024, 256, 300) for n in (512, 1024, 300) for k in (65536, 1 << 18, 1 << 20)
                   if size(m, n, k) > 0)
    a, b = _q(rows=M, cols=K, ld=K // 2, ld_scale=K // 32), _q(rows=N, cols=K, ld=K // 2, ld_scale=K // 32)
    need = size(M, N, K)
    assert need % 256 == 0 and need <= 64 << 20
    assert product(a, b, ld_y=N, n=need - 1) == WORKSPACE
    assert product(a, b, ld_y=N, ws=None) == WORKSPACE
    assert product(a, b, ld_y=N, ws=FAKE + 16, n=need) == UNSUPPORTED


def _t(n=100, weight=FAKE, master=None, grad=FAKE, m=FAKE, v=FAKE, ms=None, vs=None, dtype=F32, gdtype=F32, decay=0.1):
    return tw.TwellAdamWTensorC(n, weight, master, grad, m, v, ms, vs, dtype, gdtype, decay)


def _list(*ts):
    return (tw.TwellAdamWTensorC * len(ts))(*ts)


def step(ts=None, count=None, clip=None, args=True, **kw):
    ts = _list(_t()) if ts is None else ts
    a = tw.TwellAdamWC(**{**dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, step=1, seed=0), **kw})
    return L.twell_adamw_step(ts, len(ts) if count is None else count, ctypes.byref(a) if args else None, clip, None)


BAD_TENSORS = [
    (dict(n=-1), INVALID),
    (dict(n=BIG + 1), UNSUPPORTED),
    (dict(weight=None), INVALID),
    (dict(grad=None), INVALID),
    (dict(m=None), INVALID),
    (dict(v=None), INVALID),
    (dict(ms=FAKE), INVALID),              # one scale without the other
    (dict(vs=FAKE), INVALID),
    (dict(master=FAKE), INVALID),          # fp32 weights with an fp32 copy
    (dict(dtype=3), INVALID),
    (dict(gdtype=-2), INVALID),
    (dict(decay=float("nan")), INVALID),
    (dict(decay=float("inf")), INVALID),
    (dict(weight=FAKE + 2), UNSUPPORTED),
    (dict(weight=FAKE + 1, dtype=BF16), UNSUPPORTED),
    (dict(master=FAKE + 2, dtype=BF16), UNSUPPORTED),
    (dict(grad=FAKE + 2), UNSUPPORTED),
    (dict(grad=FAKE + 1, gdtype=BF16), UNSUPPORTED),
    (dict(m=FAKE + 2), UNSUPPORTED),
    (dict(v=FAKE + 1), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", BAD_TENSORS)
def test_step_validation_of_tensors(kw, status):
    # also behind good ones: nothing has been launched by then
    assert step(_list(_t(**kw))) == status
    assert step(_list(*[_t()] * 50, _t(**kw))) == status
    assert tw.twell_last_error().startswith("tensor 50")


@pytest.mark.parametrize("kw", [
    dict(lr=-1.0), dict(lr=float("nan")), dict(lr=float("inf")), dict(eps=-1e-8), dict(eps=float("nan")),
    dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=float("nan")), dict(step=0), dict(step=-3),
    dict(count=-1), dict(args=False)])
def test_step_validation(kw):
    assert step(**kw) == INVALID


def test_step_validation_of_pointers():
    assert step(clip=FAKE + 2) == UNSUPPORTED
    assert step(lr_device=FAKE + 2) == UNSUPPORTED
    assert step(step_device=FAKE + 4) == UNSUPPORTED
    assert L.twell_adamw_step(None, 1, ctypes.byref(tw.TwellAdamWC(1e-3, 0.9, 0.99, 1e-8, 1, 0)), None, None) == INVALID


def test_steps_without_elements_launch_nothing():
    assert step(_list(), count=0) == OK
    assert step(_list(_t(n=0, weight=None, grad=None, m=None, v=None))) == OK


def grad_norm(ts=None, count=None, max_norm=1.0, out=FAKE, ws=FAKE, n=BIG):
    ts = _list(_t()) if ts is None else ts
    return L.twell_grad_norm(ts, len(ts) if count is None else count, max_norm, out, ws, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(max_norm=0.0), INVALID), (dict(max_norm=-1.0), INVALID), (dict(max_norm=float("nan")), INVALID),
    (dict(out=None), INVALID), (dict(out=FAKE + 2), UNSUPPORTED), (dict(count=-1), INVALID),
    (dict(ws=None), WORKSPACE), (dict(n=8), WORKSPACE), (dict(ws=FAKE + 16), UNSUPPORTED),
    (dict(ts=_list(_t(n=-1))), INVALID), (dict(ts=_list(_t(grad=None))), INVALID),
    (dict(ts=_list(_t(gdtype=4))), INVALID), (dict(ts=_list(_t(grad=FAKE + 2))), UNSUPPORTED)])
def test_grad_norm_validation(kw, status):
    assert grad_norm(**kw) == status


def test_grad_norm_workspace():
    size = L.twell_grad_norm_workspace_size
    assert size(_list(), 0) == 256 and size(None, 1) == 0 and size(_list(_t(n=-1)), 1) == 0
    one, many = size(_list(_t(n=1 << 30)), 1), size(_list(*[_t(n=1 << 30)] * 300), 300)
    assert 256 <= one < many


@pytest.mark.parametrize("kw,status", [
    (dict(), INVALID),                              # 32-bit states
    (dict(ms=FAKE), INVALID), (dict(ms=FAKE, vs=FAKE, m=None), INVALID), (dict(ms=FAKE, vs=FAKE, n=-1), INVALID)])
def test_states_validation(kw, status):
    out = (ctypes.c_void_p * 1)(FAKE)
    assert L.twell_adamw_states(_list(_t(**kw)), 1, BF16, out, out, None) == status
    good = _list(_t(ms=FAKE, vs=FAKE))
    assert L.twell_adamw_states(good, 1, 7, out, out, None) == INVALID
    assert L.twell_adamw_states(good, 1, F32, (ctypes.c_void_p * 1)(FAKE + 2), None, None) == UNSUPPORTED
    assert L.twell_adamw_states(good, 1, F32, None, None, None) == OK  # nothing asked for


def test_binding_refuses():
    import torch
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    rows = tw.Mx4Rows(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 16, dtype=torch.uint8), 64)
    for call in (lambda: tw.twell_quantize_mx4(x), lambda: tw.twell_dequantize_mx4(rows),
                 lambda: tw.twell_rmsnorm_mx4(x, x[0]), lambda: tw.twell_mx4_matmul(rows, rows),
                 lambda: tw.twell_grad_norm([x]), lambda: tw.twell_grad_norm([]), lambda: tw.TwellAdamW.zeros([x]),
                 lambda: tw.TwellAdamW.zeros([]), lambda: tw.TwellAdamW.zeros([x], bits=16)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        tw.twell_quantize_mx4(x.to(torch.float16))
    with pytest.raises(ValueError):
        tw.twell_quantize_mx4(x[0])


def test_c_structures_match_the_header():
    import os
    import shutil
    import subprocess
    import tempfile
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    names = {"twell_mx4": tw.TwellMx4C, "twell_adamw_tensor": tw.TwellAdamWTensorC, "twell_adamw": tw.TwellAdamWC}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "twell.h"', "int main(void) {"]
    for c, py in names.items():
        lines.append(f'printf("%zu\\n", sizeof({c}));')
        lines += [f'printf("%zu\\n", offsetof({c}, {f[0]}));' for f in py._fields_]
    lines += ["return 0; }"]
    with tempfile.TemporaryDirectory() as d:
        src = os.path.join(d, "s.c")
        open(src, "w").write("\n".join(lines))
        subprocess.run([cc, "-I", os.path.join(root, "include"), src, "-o", os.path.join(d, "s")], check=True)
        got = [int(v) for v in subprocess.run([os.path.join(d, "s")], check=True, capture_output=True).stdout.split()]
    want = []
    for py in names.values():
        want += [ctypes.sizeof(py)] + [getattr(py, f[0]).offset for f in py._fields_]
    assert got == want
