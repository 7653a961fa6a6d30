"""The binding's own checks of the microscaled operators and the optimiser, on
stand-ins: CPU tensors that call themselves GPU tensors, with the library's entry
points replaced (CPU only: no kernel is ever launched here)."""

import pytest

tw = pytest.importorskip("activation_sparse_transformer_bf16_amd")
torch = pytest.importorskip("torch")

DEVICE = torch.device("cuda:0")


class OnGpu(torch.Tensor):
    is_cuda = property(lambda self: True)
    device = property(lambda self: DEVICE)


def gpu(t):
    return t.as_subclass(OnGpu)


@pytest.fixture(autouse=True)
def calls(monkeypatch):
    """The entry points called, in place of the calls."""
    seen = []
    monkeypatch.setattr(tw, "_launch", lambda device, fn, *args: seen.append(args))
    return seen


def rows(q, scale, cols, factor=None):
    return tw.Mx4Rows(gpu(q), gpu(scale), cols, factor)


def _one_row_views():
    """(q, scale, columns) of one row whose elements do not lie next to one another."""
    q, scale = torch.zeros(1, 32, dtype=torch.uint8), torch.zeros(1, 16, dtype=torch.uint8)
    yield torch.zeros(1, 64, dtype=torch.uint8)[:, ::2], scale, 64
    yield q, torch.zeros(1, 32, dtype=torch.uint8)[:, ::2], 64
    yield torch.zeros(1, 1, dtype=torch.uint8).expand(1, 4096), torch.zeros(1, 256, dtype=torch.uint8), 8192
    yield q, torch.zeros(1, 1, dtype=torch.uint8).expand(1, 16), 64


@pytest.mark.parametrize("view", range(4))
def test_a_single_row_has_unit_stride(view, calls):
    q, scale, cols = list(_one_row_views())[view]
    bad = rows(q, scale, cols)
    x = gpu(torch.zeros(1, cols))
    factor = gpu(torch.zeros(1))
    good = rows(torch.zeros(1, cols // 2, dtype=torch.uint8), torch.zeros(1, -(-cols // 512) * 16, dtype=torch.uint8), cols)
    for call in (lambda: tw.twell_quantize_mx4(x, out=bad), lambda: tw.twell_dequantize_mx4(bad, y=x),
                 lambda: tw.twell_rmsnorm_mx4(x, x[0], h=x, y=x, q=tw.Mx4Rows(bad.q, bad.scale, cols, factor)),
                 lambda: tw.twell_mx4_matmul(bad, good, y=gpu(torch.zeros(1, 1))),
                 lambda: tw.twell_mx4_matmul(good, bad, y=gpu(torch.zeros(1, 1)))):
        with pytest.raises(ValueError, match="unit stride"):
            call()
    assert not calls


def test_a_single_row_of_any_row_stride(calls):
    # a row's own stride to the next one says nothing where there is none; a single byte has no stride along
    wide = torch.zeros(3, 40, dtype=torch.uint8)
    one = rows(wide[1:2, :32], torch.zeros(1, 16, dtype=torch.uint8).as_strided((1, 16), (7, 1)), 64)
    tw.twell_quantize_mx4(gpu(torch.zeros(1, 64)), out=one)
    byte = rows(torch.zeros(1, 16, dtype=torch.uint8).as_strided((1, 1), (16, 5)), torch.zeros(1, 16, dtype=torch.uint8), 2)
    tw.twell_quantize_mx4(gpu(torch.zeros(1, 2)), out=byte)
    assert len(calls) == 2


def test_the_sizes_of_rows_are_fixed(calls):
    # the library's rows lie in one buffer of exactly that many
    made = tw.Mx4Rows.empty(3, 64, "cpu")
    given = rows(torch.zeros(3, 32, dtype=torch.uint8), torch.zeros(3, 16, dtype=torch.uint8), 64)
    for r in (made, given):
        for name in ("rows", "cols", "q", "scale", "factor"):
            with pytest.raises(AttributeError):
                setattr(r, name, 1000)
        assert (r.rows, r.cols) == (3, 64) and r.q.shape == (3, 32) and r.scale.shape == (3, 16)
