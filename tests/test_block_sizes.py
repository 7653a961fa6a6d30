"""Sizes that do not fit the library's 32-bit integers are refused by the
binding of the block operators, never passed on with their upper bits lost
(CPU only: stand-ins with a tensor's attributes, no kernel is launched)."""

import pytest

tw = pytest.importorskip("activation_sparse_transformer_bf16_amd")


class _Tensor:
    """A contiguous device tensor's attributes, at an address that is never dereferenced."""

    is_cuda = True

    def __init__(self, shape, dtype, device):
        self.shape, self.dtype, self.device = shape, dtype, device

    def dim(self):
        return len(self.shape)

    def stride(self):
        return (self.shape[1], 1)

    def is_contiguous(self):
        return True

    def storage_offset(self):
        return 0

    def data_ptr(self):
        return 0x100000


class _Device:
    index = 0


@pytest.fixture
def make(monkeypatch):
    import torch
    monkeypatch.setattr(tw, "_raw_stream", lambda device: 0)
    device = _Device()
    return lambda *shape, dtype=torch.bfloat16: _Tensor(shape, dtype, device)


# The low 32 bits of 2^32 are 0 rows: where nothing is refused, the call
# launches nothing and hands back whatever the outputs held.
@pytest.mark.parametrize("rows", [1 << 32, (1 << 32) + (1 << 31), 1 << 31])
def test_rows_beyond_32_bits(make, rows):
    import torch
    x, w = make(rows, 8), make(8)
    with pytest.raises(ValueError, match="exceed"):
        tw.twell_rmsnorm(x, w, y=x)
    with pytest.raises(ValueError, match="exceed"):
        tw.twell_rmsnorm_backward(x, x, w, dx=x, dweight=make(8, dtype=torch.float32))
    q, scale = make(rows, 16, dtype=torch.int8), make(rows, dtype=torch.float32)
    with pytest.raises(ValueError, match="exceed"):
        tw.twell_quantize_rows(make(rows, 16), q=q, scale=scale)
    none, s0 = make(0, 16, dtype=torch.int8), make(0, dtype=torch.float32)
    with pytest.raises(ValueError, match="exceed"):
        tw.twell_int8_matmul(q, scale, none, s0, y=make(rows, 0))
    with pytest.raises(ValueError, match="exceed"):
        tw.twell_int8_matmul(none, s0, q, scale, y=make(0, rows))


def test_columns_beyond_32_bits(make):
    import torch
    d = (1 << 32) + 8
    x = make(0, d)
    with pytest.raises(ValueError, match="exceed"):
        tw.twell_rmsnorm(x, make(d), y=x)
    with pytest.raises(ValueError, match="exceed"):
        tw.twell_quantize_rows(x, q=make(0, d, dtype=torch.int8), scale=make(0, dtype=torch.float32))
    q, s = make(0, d, dtype=torch.int8), make(0, dtype=torch.float32)
    with pytest.raises(ValueError, match="exceed"):
        tw.twell_int8_matmul(q, s, q, s, y=make(0, 0))


def test_workspace_sizes_beyond_32_bits():
    import torch
    big = 1 << 32
    assert tw.twell_int8_matmul_workspace_size(40, 515, 40000) > 0
    for M, N, K in [(big + 40, 515, 40000), (40, big + 515, 40000), (40, 515, big + 40000)]:
        assert tw.twell_int8_matmul_workspace_size(M, N, K) == 0
    assert tw.twell_rmsnorm_backward_workspace_size(big + 4, 64, torch.float32) == 0
    assert tw.twell_rmsnorm_backward_workspace_size(4, big + 64, torch.float32) == 0
