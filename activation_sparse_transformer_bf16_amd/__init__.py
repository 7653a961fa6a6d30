"""Python binding of libtwell.so, the MI355X TwELL sparse-FFN library.

Thin ctypes marshalling over the C ABI declared in ``include/twell.h``: torch
tensors supply device memory and the current HIP stream; every step of the
computation runs in the library's HIP kernels.  The functions carry the same
names as the C entry points.  Importing this package fails loudly when the
library has not been built (``python activation_sparse_transformer_bf16_amd/build.py``).
"""

from __future__ import annotations

import bisect
import ctypes
import functools
import itertools
import operator
import os
import struct
from dataclasses import dataclass
from typing import NamedTuple, Optional, Tuple

_HERE = os.path.dirname(os.path.abspath(__file__))
# TWELL_LIBRARY names another build of the same library (the host-sanitizer
# build of build.py); by default the in-tree libtwell.so.
LIB_PATH = os.environ.get("TWELL_LIBRARY") or os.path.join(_HERE, "libtwell.so")

TWELL_OK, TWELL_ERR_INVALID_ARG, TWELL_ERR_UNSUPPORTED, TWELL_ERR_WORKSPACE, TWELL_ERR_HIP = range(5)
ABI_VERSION = 3  # TWELL_ABI_VERSION of include/twell.h that these mirrors follow
TWELL_F32, TWELL_BF16 = 0, 1
TWELL_LAYOUT_ROWS, TWELL_LAYOUT_TILES = 0, 1


class TwellMatrixC(ctypes.Structure):
    """Mirror of ``twell_matrix`` (include/twell.h)."""

    _fields_ = [
        ("rows", ctypes.c_int32), ("cols", ctypes.c_int32), ("tile", ctypes.c_int32),
        ("cap", ctypes.c_int32), ("dtype", ctypes.c_int), ("cnt", ctypes.c_void_p),
        ("val", ctypes.c_void_p), ("idx", ctypes.c_void_p), ("ovf_rows", ctypes.c_void_p),
        ("n_ovf", ctypes.c_void_p), ("dense", ctypes.c_void_p), ("ovf_cap", ctypes.c_int32),
        ("u", ctypes.c_void_p), ("layout", ctypes.c_int),
    ]


LAYOUTS = {"rows": TWELL_LAYOUT_ROWS, "tiles": TWELL_LAYOUT_TILES}  # twell_layout: record (t, k) at t * nt + k, or at k * rows + t


class TwellHybridC(ctypes.Structure):
    """Mirror of ``twell_hybrid`` (include/twell.h)."""

    _fields_ = [
        ("rows", ctypes.c_int32), ("cols", ctypes.c_int32), ("width", ctypes.c_int32),
        ("dtype", ctypes.c_int), ("cnt", ctypes.c_void_p), ("val", ctypes.c_void_p),
        ("col", ctypes.c_void_p), ("dense_rows", ctypes.c_void_p), ("n_dense", ctypes.c_void_p),
        ("dense", ctypes.c_void_p), ("dense_cap", ctypes.c_int32), ("u", ctypes.c_void_p),
    ]


class TwellInt8C(ctypes.Structure):
    """Mirror of ``twell_int8`` (include/twell.h)."""

    _fields_ = [
        ("rows", ctypes.c_int32), ("cols", ctypes.c_int32), ("ld", ctypes.c_int64),
        ("q", ctypes.c_void_p), ("scale", ctypes.c_void_p),
    ]


class TwellMx4C(ctypes.Structure):
    """Mirror of ``twell_mx4`` (include/twell.h)."""

    _fields_ = [
        ("rows", ctypes.c_int32), ("cols", ctypes.c_int32), ("ld", ctypes.c_int64), ("q", ctypes.c_void_p),
        ("ld_scale", ctypes.c_int64), ("scale", ctypes.c_void_p), ("factor", ctypes.c_void_p),
    ]


class TwellAdamWTensorC(ctypes.Structure):
    """Mirror of ``twell_adamw_tensor`` (include/twell.h)."""

    _fields_ = [
        ("n", ctypes.c_int64), ("weight", ctypes.c_void_p), ("master", ctypes.c_void_p), ("grad", ctypes.c_void_p),
        ("m", ctypes.c_void_p), ("v", ctypes.c_void_p), ("m_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
        ("dtype", ctypes.c_int), ("grad_dtype", ctypes.c_int), ("weight_decay", ctypes.c_float),
    ]


class TwellAdamWC(ctypes.Structure):
    """Mirror of ``twell_adamw`` (include/twell.h)."""

    _fields_ = [
        ("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("eps", ctypes.c_double),
        ("step", ctypes.c_int64), ("seed", ctypes.c_uint64), ("lr_device", ctypes.c_void_p),
        ("step_device", ctypes.c_void_p),
    ]


class TwellError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{message} (status {status})")
        self.status = status


def _load():
    # torch ships its own libamdhip64.so.7; importing it first makes libtwell.so
    # bind to that same HIP runtime instead of loading a second one.
    import torch  # noqa: F401
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python activation_sparse_transformer_bf16_amd/build.py`")
    lib = ctypes.CDLL(LIB_PATH)
    lib.twell_abi_version.restype = ctypes.c_int
    if lib.twell_abi_version() != ABI_VERSION:
        raise ImportError(f"{LIB_PATH} has ABI version {lib.twell_abi_version()}, this binding needs {ABI_VERSION}: "
                          "rebuild it")
    P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    L, R = ctypes.c_int64, ctypes.c_float
    M, Q = ctypes.POINTER(TwellMatrixC), ctypes.POINTER(TwellInt8C)
    X = ctypes.POINTER(TwellMx4C)
    sig = {
        "twell_abi_version": (I, []),
        "twell_status_str": (ctypes.c_char_p, [I]),
        "twell_last_error": (ctypes.c_char_p, []),
        "twell_pack": (I, [P, M, P]),
        "twell_ffn_workspace_size": (Z, [I, I, I, I, I, I]),
        "twell_ffn_forward": (I, [P, P, P, P, P, P, I, M, P, Z, P]),
        "twell_ffn_forward_noalloc": (I, [P, P, P, P, P, P, I, M, P]),
        "twell_gate_pack": (I, [P, P, P, I, M, P, P]),
        "twell_overflow_scan": (I, [M, P]),
        "twell_sparse_ffn": (I, [M, P, P, P, P, P, P, I, P, Z, P]),
        "twell_sparse_ffn_fused": (I, [M, P, P, P, P, P, P, I, P, Z, P]),
        "twell_sparse_ffn_grouped": (I, [M, P, P, P, P, P, P, I, P, Z, P]),
        "twell_sparse_ffn_grouped_workspace_size": (Z, [I, I, I, I, I, I]),
        "dense_ffn_workspace_size": (Z, [I, I, I, I]),
        "dense_ffn_forward": (I, [P, P, P, P, P, P, I, I, I, I, P, Z, P]),
        "twell_to_hybrid": (I, [M, ctypes.POINTER(TwellHybridC), P]),
        "twell_l1_workspace_size": (Z, []),
        "twell_l1_norm": (I, [M, P, P, Z, P]),
        "twell_l1_grad": (I, [M, ctypes.c_float, P, P, P]),
        "twell_ffn_backward_workspace_size": (Z, [I, I, I, I, I, I]),
        "twell_stream_probe": (I, [P, P, Z, I, P]),
        "twell_mfma_probe": (I, [P, I, I, P]),
        "twell_ffn_backward": (I, [ctypes.POINTER(TwellHybridC), P, P, P, P, P, ctypes.c_float, I, P, P, P, P,
                                   P, Z, P]),
        "twell_rmsnorm": (I, [P, L, P, L, P, R, I, I, I, P, L, P, L, Q, P]),
        "twell_rmsnorm_backward_workspace_size": (Z, [I, I, I]),
        "twell_rmsnorm_backward": (I, [P, L, P, L, P, P, L, R, I, I, I, P, L, P, P, Z, P]),
        "twell_quantize_rows": (I, [P, L, I, Q, P]),
        "twell_int8_matmul_workspace_size": (Z, [I, I, I]),
        "twell_int8_matmul": (I, [Q, Q, P, I, P, L, P, Z, P]),
        "twell_quantize_mx4": (I, [P, L, I, X, P]),
        "twell_dequantize_mx4": (I, [X, I, P, L, P]),
        "twell_rmsnorm_mx4": (I, [P, L, P, L, P, R, I, I, I, P, L, P, L, X, P]),
        "twell_mx4_matmul_workspace_size": (Z, [I, I, I]),
        "twell_mx4_matmul": (I, [X, X, P, I, P, L, P, Z, P]),
        "twell_grad_norm_workspace_size": (Z, [P, I]),
        "twell_grad_norm": (I, [P, I, R, P, P, Z, P]),
        "twell_adamw_step": (I, [P, I, ctypes.POINTER(TwellAdamWC), P, P]),
        "twell_adamw_states": (I, [P, I, I, P, P, P]),
    }
    # Private function objects: changing argtypes on the public handle (lib())
    # cannot make this binding pass truncated pointers.
    fns = {}
    for name, (res, args) in sig.items():
        for fn in (lib._FuncPtr((name, lib)), getattr(lib, name)):
            fn.restype, fn.argtypes = res, args
        fns[name] = lib._FuncPtr((name, lib))
        fns[name].restype, fns[name].argtypes = res, args
    return lib, fns


class _Fns:
    def __init__(self, fns):
        self.__dict__.update(fns)


_public_lib, _private = _load()
_lib = _Fns(_private)

import torch as _t  # noqa: E402  (loaded by _load, before the library)

_torch_c = _t._C
_INT8, _UINT8, _INT64 = _t.int8, _t.uint8, _t.int64
_FLOAT32, _BFLOAT16 = _t.float32, _t.bfloat16
_CODES = {_FLOAT32: TWELL_F32, _BFLOAT16: TWELL_BF16}
_SIZES = (4, 2)  # bytes, by code
_CONTIGUOUS = _t.contiguous_format

# Names every build of the library must export (checked by the CPU tests).
EXPORTS = ("twell_abi_version", "twell_status_str", "twell_last_error", "twell_pack",
           "twell_ffn_workspace_size", "twell_ffn_forward", "twell_gate_pack", "twell_overflow_scan",
           "twell_sparse_ffn",
           "dense_ffn_workspace_size", "dense_ffn_forward", "twell_to_hybrid",
           "twell_l1_workspace_size", "twell_l1_norm", "twell_l1_grad",
           "twell_ffn_backward_workspace_size", "twell_ffn_backward", "twell_sparse_ffn_fused",
           "twell_stream_probe", "twell_mfma_probe", "twell_ffn_forward_noalloc", "twell_sparse_ffn_grouped",
           "twell_sparse_ffn_grouped_workspace_size",
           "twell_rmsnorm", "twell_rmsnorm_backward_workspace_size", "twell_rmsnorm_backward",
           "twell_quantize_rows", "twell_int8_matmul_workspace_size", "twell_int8_matmul",
           "twell_quantize_mx4", "twell_dequantize_mx4", "twell_rmsnorm_mx4", "twell_mx4_matmul_workspace_size",
           "twell_mx4_matmul", "twell_grad_norm_workspace_size", "twell_grad_norm", "twell_adamw_step",
           "twell_adamw_states")

# Size of the static device scratch behind twell_ffn_forward_noalloc
# (TWELL_NOALLOC_SCRATCH_BYTES in include/twell.h).
NOALLOC_SCRATCH_BYTES = 64 << 20


def lib():
    """The ctypes handle of libtwell.so (its functions have argtypes set)."""
    return _public_lib


def twell_abi_version() -> int:
    return _lib.twell_abi_version()


def twell_status_str(status: int) -> str:
    return _lib.twell_status_str(status).decode()


def twell_last_error() -> str:
    return _lib.twell_last_error().decode()


def _check(status: int):
    if status != TWELL_OK:
        raise TwellError(status, f"{twell_status_str(status)}: {twell_last_error()}")


# --------------------------------------------------------------------------- torch glue

def _torch():
    import torch
    return torch


def _dtype_code(t) -> int:
    torch = _torch()
    if t == torch.float32:
        return TWELL_F32
    if t == torch.bfloat16:
        return TWELL_BF16
    raise TypeError(f"unsupported dtype {t} (float32 or bfloat16)")


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(device) -> int:
    torch = _torch()
    return torch.cuda.current_stream(device).cuda_stream


def _need(t, name, device, dtype=None, shape=None):
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


@dataclass
class TwellMatrix:
    """Device buffers of one TwELL matrix (see ``twell_matrix`` in include/twell.h)."""

    rows: int
    cols: int
    tile: int
    cap: int
    dtype: object        # torch dtype of the values
    cnt: object          # int16 [rows, cols/tile] (uint16 bit patterns); tile-major: [cols/tile, rows]
    val: object          # dtype [rows, cols/tile, cap]; tile-major: [cols/tile, rows, cap]
    idx: object          # uint8 [rows, cols/tile, cap]; tile-major: [cols/tile, rows, cap]
    ovf_rows: object     # int32 [ovf_cap]
    n_ovf: object        # int32 [1]
    dense: object        # dtype [ovf_cap, cols] or None
    ovf_cap: int
    u: object = None     # float32 [rows, cols/tile, cap] (u saved by the forward) or None
    layout: str = "rows"  # "rows" (row-major records) or "tiles" (tile-major, see twell_matrix)

    @classmethod
    def empty(cls, rows: int, cols: int, tile: int, cap: int, dtype, device,
              ovf_cap: Optional[int] = None, dense: bool = True, u: bool = False,
              layout: str = "rows") -> "TwellMatrix":
        torch = _torch()
        nt = cols // tile
        ovf_cap = rows if ovf_cap is None else ovf_cap
        if layout not in LAYOUTS:
            raise ValueError(f"layout must be one of {sorted(LAYOUTS)}, got {layout!r}")
        r2 = (rows, nt) if layout == "rows" else (nt, rows)
        return cls(rows, cols, tile, cap, dtype,
                   torch.empty(r2, dtype=torch.int16, device=device),
                   torch.empty(r2 + (cap,), dtype=dtype, device=device),
                   torch.empty(r2 + (cap,), dtype=torch.uint8, device=device),
                   torch.empty((max(ovf_cap, 1),), dtype=torch.int32, device=device),
                   torch.empty((1,), dtype=torch.int32, device=device),
                   torch.empty((max(ovf_cap, 1), cols), dtype=dtype, device=device) if dense else None,
                   ovf_cap,
                   torch.empty(r2 + (cap,), dtype=torch.float32, device=device) if u else None,
                   layout)

    def validate(self, device=None) -> None:
        """Check every buffer against the matrix's own fields (device, dtype,
        shape, contiguity) before its pointers reach the library."""
        torch = _torch()
        device = self.cnt.device if device is None else device
        _dtype_code(self.dtype)
        if self.rows < 0 or self.cols <= 0 or self.tile <= 0 or self.cap <= 0 or self.cols % self.tile:
            raise ValueError(f"bad TwELL shape rows={self.rows} cols={self.cols} tile={self.tile} cap={self.cap}")
        nt = self.cols // self.tile
        if self.layout not in LAYOUTS:
            raise ValueError(f"layout must be one of {sorted(LAYOUTS)}, got {self.layout!r}")
        r2 = (self.rows, nt) if self.layout == "rows" else (nt, self.rows)
        _need(self.cnt, "cnt", device, torch.int16, r2)
        _need(self.val, "val", device, self.dtype, r2 + (self.cap,))
        _need(self.idx, "idx", device, torch.uint8, r2 + (self.cap,))
        _need(self.ovf_rows, "ovf_rows", device, torch.int32)
        if self.ovf_rows.numel() < max(self.ovf_cap, 1):
            raise ValueError(f"ovf_rows holds {self.ovf_rows.numel()} entries, ovf_cap is {self.ovf_cap}")
        _need(self.n_ovf, "n_ovf", device, torch.int32, (1,))
        if self.dense is not None:
            _need(self.dense, "dense", device, self.dtype)
            if self.dense.dim() != 2 or self.dense.shape[1] != self.cols or self.dense.shape[0] < self.ovf_cap:
                raise ValueError(f"dense must have shape (>= {self.ovf_cap}, {self.cols}), "
                                 f"got {tuple(self.dense.shape)}")
        if self.u is not None:
            _need(self.u, "u", device, torch.float32, r2 + (self.cap,))

    def c_struct(self) -> TwellMatrixC:
        return TwellMatrixC(self.rows, self.cols, self.tile, self.cap, _dtype_code(self.dtype),
                            _ptr(self.cnt), _ptr(self.val), _ptr(self.idx), _ptr(self.ovf_rows),
                            _ptr(self.n_ovf), _ptr(self.dense), self.ovf_cap, _ptr(self.u),
                            LAYOUTS.get(self.layout, -1))

    @property
    def device(self):
        return self.cnt.device


@dataclass
class TwellHybrid:
    """Device buffers of one hybrid matrix (see ``twell_hybrid`` in include/twell.h)."""

    rows: int
    cols: int
    width: int
    dtype: object        # torch dtype of the values
    cnt: object          # int32 [rows]
    val: object          # dtype [rows, width]
    col: object          # int32 [rows, width]
    dense_rows: object   # int32 [dense_cap]
    n_dense: object      # int32 [1]
    dense: object        # dtype [dense_cap, cols] or None
    dense_cap: int
    u: object = None     # float32 [rows, width] (saved u of the ELL slots) or None

    @classmethod
    def empty(cls, rows: int, cols: int, width: int, dtype, device, dense_cap: Optional[int] = None,
              dense: bool = True, u: bool = False) -> "TwellHybrid":
        torch = _torch()
        dense_cap = rows if dense_cap is None else dense_cap
        return cls(rows, cols, width, dtype,
                   torch.empty((rows,), dtype=torch.int32, device=device),
                   torch.empty((rows, width), dtype=dtype, device=device),
                   torch.empty((rows, width), dtype=torch.int32, device=device),
                   torch.empty((max(dense_cap, 1),), dtype=torch.int32, device=device),
                   torch.empty((1,), dtype=torch.int32, device=device),
                   torch.empty((max(dense_cap, 1), cols), dtype=dtype, device=device) if dense else None,
                   dense_cap,
                   torch.empty((rows, width), dtype=torch.float32, device=device) if u else None)

    def validate(self, device=None) -> None:
        """Check every buffer against the hybrid matrix's own fields."""
        torch = _torch()
        device = self.cnt.device if device is None else device
        _dtype_code(self.dtype)
        if self.rows < 0 or self.cols <= 0 or self.width < 1 or self.dense_cap < 0:
            raise ValueError(f"bad hybrid shape rows={self.rows} cols={self.cols} width={self.width}")
        _need(self.cnt, "cnt", device, torch.int32, (self.rows,))
        _need(self.val, "val", device, self.dtype, (self.rows, self.width))
        _need(self.col, "col", device, torch.int32, (self.rows, self.width))
        _need(self.dense_rows, "dense_rows", device, torch.int32)
        if self.dense_rows.numel() < max(self.dense_cap, 1):
            raise ValueError(f"dense_rows holds {self.dense_rows.numel()} entries, dense_cap is {self.dense_cap}")
        _need(self.n_dense, "n_dense", device, torch.int32, (1,))
        if self.dense is not None:
            _need(self.dense, "dense", device, self.dtype)
            if self.dense.dim() != 2 or self.dense.shape[1] != self.cols or self.dense.shape[0] < self.dense_cap:
                raise ValueError(f"dense must have shape (>= {self.dense_cap}, {self.cols}), "
                                 f"got {tuple(self.dense.shape)}")
        if self.u is not None:
            _need(self.u, "u", device, torch.float32, (self.rows, self.width))

    def c_struct(self) -> TwellHybridC:
        return TwellHybridC(self.rows, self.cols, self.width, _dtype_code(self.dtype), _ptr(self.cnt),
                            _ptr(self.val), _ptr(self.col), _ptr(self.dense_rows), _ptr(self.n_dense),
                            _ptr(self.dense), self.dense_cap, _ptr(self.u))


def twell_to_hybrid(packed: TwellMatrix, width: int, dense_cap: Optional[int] = None, dense: bool = True,
                    out: Optional[TwellHybrid] = None) -> TwellHybrid:
    """Convert a TwELL matrix (with its dense backup rows) to the hybrid format;
    a new ``out`` carries the saved u when the TwELL matrix has one."""
    packed.validate()
    if out is None:
        out = TwellHybrid.empty(packed.rows, packed.cols, width, packed.dtype, packed.device, dense_cap, dense,
                                u=packed.u is not None)
    out.validate(packed.device)
    if (out.rows, out.cols, out.width, out.dtype) != (packed.rows, packed.cols, width, packed.dtype):
        raise ValueError("out must be a hybrid matrix of the TwELL matrix's rows, cols and dtype at this width")
    m = packed.c_struct()
    h = out.c_struct()
    _check(_lib.twell_to_hybrid(ctypes.byref(m), ctypes.byref(h), _stream(packed.device)))
    return out


def twell_l1_workspace_size() -> int:
    return int(_lib.twell_l1_workspace_size())


def twell_l1_norm(packed: TwellMatrix, out=None, workspace=None):
    """||h||_1 of the activations a TwELL matrix describes, as a float64 device tensor [1]."""
    torch = _torch()
    device = packed.device
    packed.validate()
    if out is None:
        out = torch.empty((1,), dtype=torch.float64, device=device)
    _need(out, "out", device, torch.float64, (1,))
    ws = _workspace(twell_l1_workspace_size(), device, workspace)
    m = packed.c_struct()
    _check(_lib.twell_l1_norm(ctypes.byref(m), _ptr(out), _ptr(ws), ws.numel(), _stream(device)))
    return out


def twell_l1_grad(packed: TwellMatrix, lam: float, grad_val=None, grad_dense=None, dense: bool = True):
    """d(lam ||h||_1)/dh in the TwELL pattern: (grad_val, grad_dense or None)."""
    torch = _torch()
    device = packed.device
    packed.validate()
    if grad_val is None:
        grad_val = torch.empty_like(packed.val)
    if grad_dense is None and dense and packed.dense is not None:
        grad_dense = torch.empty_like(packed.dense)
    _need(grad_val, "grad_val", device, packed.dtype, tuple(packed.val.shape))
    if grad_dense is not None:
        if packed.dense is None:
            raise ValueError("grad_dense needs the TwELL matrix's dense backup rows")
        _need(grad_dense, "grad_dense", device, packed.dtype, tuple(packed.dense.shape))
    m = packed.c_struct()
    _check(_lib.twell_l1_grad(ctypes.byref(m), ctypes.c_float(lam), _ptr(grad_val), _ptr(grad_dense),
                              _stream(device)))
    return grad_val, grad_dense


def twell_ffn_backward_workspace_size(T: int, d: int, F: int, width: int, dense_cap: int, dtype) -> int:
    return int(_lib.twell_ffn_backward_workspace_size(T, d, F, width, dense_cap, _dtype_code(dtype)))


def twell_ffn_backward(hy: TwellHybrid, x, w_gate, w_up, w_down, dy, lam: float = 0.0, dx=None, dw_gate=None,
                       dw_up=None, dw_down=None, workspace=None):
    """Gradients of the FFN layer from its hybrid activations: (dx, dw_gate, dw_up, dw_down);
    dx in the activation dtype, the weight gradients fp32 [F, d]."""
    torch = _torch()
    device = x.device
    T, d = x.shape
    F = hy.cols
    hy.validate(device)
    _need(x, "x", device, hy.dtype, (hy.rows, d))
    _need(dy, "dy", device, hy.dtype, (T, d))
    for w, name in ((w_gate, "w_gate"), (w_up, "w_up"), (w_down, "w_down")):
        _need(w, name, device, hy.dtype, (F, d))
    if dx is None:
        dx = torch.empty((T, d), dtype=hy.dtype, device=device)
    outs = []
    for g, name in ((dw_gate, "dw_gate"), (dw_up, "dw_up"), (dw_down, "dw_down")):
        if g is None:
            g = torch.empty((F, d), dtype=torch.float32, device=device)
        _need(g, name, device, torch.float32, (F, d))
        outs.append(g)
    _need(dx, "dx", device, hy.dtype, (T, d))
    ws = _workspace(twell_ffn_backward_workspace_size(T, d, F, hy.width, hy.dense_cap, hy.dtype), device,
                    workspace)
    h = hy.c_struct()
    _check(_lib.twell_ffn_backward(ctypes.byref(h), _ptr(x), _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(dy),
                                   ctypes.c_float(lam), d, _ptr(dx), _ptr(outs[0]), _ptr(outs[1]), _ptr(outs[2]),
                                   _ptr(ws), ws.numel(), _stream(device)))
    return dx, outs[0], outs[1], outs[2]


def twell_pack(pre, tile: int, cap: int, ovf_cap: Optional[int] = None, dense: bool = True,
               out: Optional[TwellMatrix] = None) -> TwellMatrix:
    """Pack a pre-activation matrix [T, F] (fp32 or bf16, on the GPU) into TwELL."""
    device = pre.device
    _need(pre, "pre", device)
    _dtype_code(pre.dtype)
    if pre.dim() != 2:
        raise ValueError(f"pre must be 2-D [T, F], got shape {tuple(pre.shape)}")
    T, F = pre.shape
    if out is None:
        out = TwellMatrix.empty(T, F, tile, cap, pre.dtype, device, ovf_cap, dense)
    out.validate(device)
    if (out.rows, out.cols, out.tile, out.cap, out.dtype) != (T, F, tile, cap, pre.dtype):
        raise ValueError(f"out ({out.rows}x{out.cols}, tile {out.tile}, cap {out.cap}, {out.dtype}) does not "
                         f"match pre ({T}x{F}, {pre.dtype}) at tile {tile}, cap {cap}")
    m = out.c_struct()
    _check(_lib.twell_pack(_ptr(pre), ctypes.byref(m), _stream(device)))
    return out


def twell_ffn_workspace_size(T: int, d: int, F: int, tile: int, cap: int, dtype) -> int:
    return int(_lib.twell_ffn_workspace_size(T, d, F, tile, cap, _dtype_code(dtype)))


def dense_ffn_workspace_size(T: int, d: int, F: int, dtype) -> int:
    return int(_lib.dense_ffn_workspace_size(T, d, F, _dtype_code(dtype)))


def _ffn_checks(x, w_gate, w_up, w_down, gate_bias):
    torch = _torch()
    device = x.device
    if x.dim() != 2 or w_gate.dim() != 2:
        raise ValueError("x and the weights must be 2-D")
    T, d = x.shape
    F = w_gate.shape[0]
    _need(x, "x", device)
    _dtype_code(x.dtype)
    for name, w in (("w_gate", w_gate), ("w_up", w_up), ("w_down", w_down)):
        _need(w, name, device, x.dtype, (F, d))
    if gate_bias is not None:
        _need(gate_bias, "gate_bias", device, torch.float32, (T,))
    return device, T, d, F


def _workspace(nbytes: int, device, workspace=None):
    torch = _torch()
    if workspace is not None:
        _need(workspace, "workspace", device, torch.uint8)
        if workspace.numel() >= nbytes:
            return workspace
    return torch.empty((max(nbytes, 1),), dtype=torch.uint8, device=device)


def _packed_for(packed: TwellMatrix, device, T: int, F: int, dtype) -> None:
    """A caller's TwELL matrix must describe exactly the activations of x."""
    packed.validate(device)
    if (packed.rows, packed.cols, packed.dtype) != (T, F, dtype):
        raise ValueError(f"packed ({packed.rows}x{packed.cols}, {packed.dtype}) does not match the layer "
                         f"({T} tokens x {F} units, {dtype})")


def twell_ffn_forward(x, w_gate, w_up, w_down, gate_bias=None, tile: int = 256, cap: int = 16,
                      packed: Optional[TwellMatrix] = None, y=None, workspace=None
                      ) -> Tuple[object, TwellMatrix]:
    """y = (ReLU(x W_g^T + beta) * (x W_u^T)) W_d through TwELL; returns (y, packed)."""
    torch = _torch()
    device, T, d, F = _ffn_checks(x, w_gate, w_up, w_down, gate_bias)
    if packed is None:
        packed = TwellMatrix.empty(T, F, tile, cap, x.dtype, device, T, dense=False)
    _packed_for(packed, device, T, F, x.dtype)
    if y is None:
        y = torch.empty((T, d), dtype=x.dtype, device=device)
    _need(y, "y", device, x.dtype, (T, d))
    ws = _workspace(twell_ffn_workspace_size(T, d, F, packed.tile, packed.cap, x.dtype), device, workspace)
    m = packed.c_struct()
    _check(_lib.twell_ffn_forward(_ptr(x), _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(gate_bias),
                                  _ptr(y), d, ctypes.byref(m), _ptr(ws),
                                  ws.numel(), _stream(device)))
    return y, packed


def twell_ffn_forward_noalloc(x, w_gate, w_up, w_down, packed: TwellMatrix, y, gate_bias=None):
    """twell_ffn_forward with its workspace in the library's static device
    scratch: the caller passes the outputs (packed, y) and nothing is
    allocated.  Calls that overlap on one GPU race (one scratch per GPU)."""
    device, T, d, F = _ffn_checks(x, w_gate, w_up, w_down, gate_bias)
    _packed_for(packed, device, T, F, x.dtype)
    _need(y, "y", device, x.dtype, (T, d))
    m = packed.c_struct()
    _check(_lib.twell_ffn_forward_noalloc(_ptr(x), _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(gate_bias),
                                          _ptr(y), d, ctypes.byref(m), _stream(device)))
    return y, packed


def twell_gate_pack(x, w_gate, gate_bias=None, tile: int = 256, cap: int = 16,
                    packed: Optional[TwellMatrix] = None, pre_out: bool = False, scan: bool = True):
    """Gate matmul + TwELL epilogue (one kernel), then, with ``scan``, the overflow
    scan; returns (packed, pre or None)."""
    torch = _torch()
    device = x.device
    if x.dim() != 2 or w_gate.dim() != 2:
        raise ValueError("x and w_gate must be 2-D")
    T, d = x.shape
    F = w_gate.shape[0]
    _need(x, "x", device)
    _dtype_code(x.dtype)
    _need(w_gate, "w_gate", device, x.dtype, (F, d))
    if gate_bias is not None:
        _need(gate_bias, "gate_bias", device, torch.float32, (T,))
    if packed is None:
        packed = TwellMatrix.empty(T, F, tile, cap, x.dtype, device, T, dense=False)
    _packed_for(packed, device, T, F, x.dtype)
    pre = torch.empty((T, F), dtype=x.dtype, device=device) if pre_out else None
    m = packed.c_struct()
    _check(_lib.twell_gate_pack(_ptr(x), _ptr(w_gate), _ptr(gate_bias), d, ctypes.byref(m),
                                _ptr(pre), _stream(device)))
    if scan:
        twell_overflow_scan(packed)
    return packed, pre


def twell_overflow_scan(packed: TwellMatrix) -> TwellMatrix:
    """List the overflowing rows of a packed matrix (fills ovf_rows and n_ovf)."""
    packed.validate()
    m = packed.c_struct()
    _check(_lib.twell_overflow_scan(ctypes.byref(m), _stream(packed.device)))
    return packed


def twell_sparse_ffn(packed: TwellMatrix, x, w_gate, w_up, w_down, gate_bias=None, y=None,
                     workspace=None):
    """Up / down projections over TwELL plus the dense fallback; returns y."""
    torch = _torch()
    device, T, d, F = _ffn_checks(x, w_gate, w_up, w_down, gate_bias)
    _packed_for(packed, device, T, F, x.dtype)
    if y is None:
        y = torch.empty((T, d), dtype=x.dtype, device=device)
    _need(y, "y", device, x.dtype, (T, d))
    ws = _workspace(twell_ffn_workspace_size(T, d, F, packed.tile, packed.cap, x.dtype), device, workspace)
    m = packed.c_struct()
    _check(_lib.twell_sparse_ffn(ctypes.byref(m), _ptr(x), _ptr(w_gate), _ptr(w_up), _ptr(w_down),
                                 _ptr(gate_bias), _ptr(y), d, _ptr(ws), ws.numel(),
                                 _stream(device)))
    return y


def twell_sparse_ffn_fused(packed: TwellMatrix, x, w_gate, w_up, w_down, gate_bias=None, y=None,
                           workspace=None):
    """twell_sparse_ffn with the up and down projections in one kernel; returns y."""
    torch = _torch()
    device, T, d, F = _ffn_checks(x, w_gate, w_up, w_down, gate_bias)
    _packed_for(packed, device, T, F, x.dtype)
    if y is None:
        y = torch.empty((T, d), dtype=x.dtype, device=device)
    _need(y, "y", device, x.dtype, (T, d))
    ws = _workspace(twell_ffn_workspace_size(T, d, F, packed.tile, packed.cap, x.dtype), device, workspace)
    m = packed.c_struct()
    _check(_lib.twell_sparse_ffn_fused(ctypes.byref(m), _ptr(x), _ptr(w_gate), _ptr(w_up), _ptr(w_down),
                                       _ptr(gate_bias), _ptr(y), d, _ptr(ws), ws.numel(), _stream(device)))
    return y


def twell_sparse_ffn_grouped_workspace_size(T: int, d: int, F: int, tile: int, cap: int, dtype) -> int:
    return int(_lib.twell_sparse_ffn_grouped_workspace_size(T, d, F, tile, cap, _dtype_code(dtype)))


def twell_sparse_ffn_grouped(packed: TwellMatrix, x, w_gate, w_up, w_down, gate_bias=None, y=None,
                             workspace=None):
    """twell_sparse_ffn with the fused up+down kernel in hidden-group-major order
    (fp32 partial output rows per group, added in group order); returns y."""
    torch = _torch()
    device, T, d, F = _ffn_checks(x, w_gate, w_up, w_down, gate_bias)
    _packed_for(packed, device, T, F, x.dtype)
    if y is None:
        y = torch.empty((T, d), dtype=x.dtype, device=device)
    _need(y, "y", device, x.dtype, (T, d))
    ws = _workspace(twell_sparse_ffn_grouped_workspace_size(T, d, F, packed.tile, packed.cap, x.dtype), device,
                    workspace)
    m = packed.c_struct()
    _check(_lib.twell_sparse_ffn_grouped(ctypes.byref(m), _ptr(x), _ptr(w_gate), _ptr(w_up), _ptr(w_down),
                                         _ptr(gate_bias), _ptr(y), d, _ptr(ws), ws.numel(), _stream(device)))
    return y


def dense_ffn_forward(x, w_gate, w_up, w_down, gate_bias=None, y=None, workspace=None):
    """The same layer computed densely on the matrix cores (baseline)."""
    torch = _torch()
    device, T, d, F = _ffn_checks(x, w_gate, w_up, w_down, gate_bias)
    if y is None:
        y = torch.empty((T, d), dtype=x.dtype, device=device)
    _need(y, "y", device, x.dtype, (T, d))
    ws = _workspace(dense_ffn_workspace_size(T, d, F, x.dtype), device, workspace)
    _check(_lib.dense_ffn_forward(_ptr(x), _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(gate_bias),
                                  _ptr(y), T, d, F, _dtype_code(x.dtype), _ptr(ws), ws.numel(),
                                  _stream(device)))
    return y


# --------------------------------------------------------------------------- block operators

class RmsNormOut(NamedTuple):
    """What ``twell_rmsnorm`` wrote (None: not asked for); ``h`` is x itself without a residual."""

    y: object       # dtype [rows, d]
    h: object       # dtype [rows, d]
    q: object       # int8 [rows, d], rows 16-byte aligned
    scale: object   # float32 [rows]


# A decoding step calls these operators with a few rows, where the kernel takes
# 2-5 us: the checks below compare first and word the error only when one
# fails, and outputs made here are not checked again.

# Sizes are 32-bit in the library, and ctypes passes the low 32 bits of a larger
# number: one that does not fit has to be refused here.
_MAX_SIZE = (1 << 31) - 1


def _bad_rows(t, name, device, dtype, shape):
    """The error of the first check that a 2-D operand fails."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.device != device or not t.is_cuda:
        raise ValueError(f"{name} must be on {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if max(shape) > _MAX_SIZE:
        raise ValueError(f"{name}: sizes of {tuple(shape)} exceed {_MAX_SIZE}")
    raise ValueError(f"{name} must have unit stride along its rows")


def _rows(t, name, device, dtype, shape) -> int:
    """Checks a 2-D tensor with unit stride along its rows; returns the row stride in elements."""
    if t is None or t.dtype != dtype or t.device != device or not t.is_cuda or t.shape != shape:
        _bad_rows(t, name, device, dtype, shape)
    rows, cols = shape
    if rows > _MAX_SIZE or cols > _MAX_SIZE:
        _bad_rows(t, name, device, dtype, shape)
    if rows == 0:
        return cols
    across, along = t.stride()
    if along != 1 and cols > 1:
        _bad_rows(t, name, device, dtype, shape)
    return across if rows > 1 else cols


def _vec(t, name, device, dtype, n) -> int:
    """Checks a contiguous vector of n elements; returns its address."""
    if t is None or t.dtype != dtype or t.device != device or t.shape != (n,) or not t.is_contiguous():
        _need(t, name, device, dtype, (n,))
    return t.data_ptr()


def _raw_stream(device) -> int:
    """The current stream's handle without building a Stream object (0.1 against 1.9 us)."""
    return _torch_c._cuda_getCurrentRawStream(device.index)


def _int8_rows(q, scale, name, device, shape) -> TwellInt8C:
    """The descriptor of int8 rows given as tensors: every row 16-byte aligned,
    with its last 16-byte chunk inside the tensor's storage."""
    ld = _rows(q, name, device, _INT8, shape)
    sp = _vec(scale, f"{name}_scale", device, _FLOAT32, shape[0])
    rows, cols = shape
    wide = (cols + 15) // 16 * 16
    if rows <= 1:
        ld = wide
    elif ld % 16:
        raise ValueError(f"{name}: row stride {ld} is not a multiple of 16 (lay rows out as twell_quantize_rows does)")
    if wide != cols and rows and q.storage_offset() + (rows - 1) * ld + wide > q.untyped_storage().nbytes():
        raise ValueError(f"{name}: the last row's 16-byte chunks run past the tensor's storage")
    return TwellInt8C(rows, cols, ld, q.data_ptr(), sp)


def _new_int8_rows(x):
    """int8 rows (16-byte aligned) and scales for the rows of x, and their descriptor."""
    rows, cols = x.shape
    ld = (cols + 15) // 16 * 16
    q = x.new_empty((rows, ld), dtype=_INT8)
    scale = x.new_empty((rows,), dtype=_FLOAT32)
    desc = TwellInt8C(rows, cols, ld, q.data_ptr(), scale.data_ptr())
    return (q if ld == cols else q[:, :cols]), scale, desc


def twell_rmsnorm(x, weight, eps: float = 1e-6, residual=None, quantize: bool = False, h=None, y=None, q=None,
                  scale=None, want_y: bool = True) -> RmsNormOut:
    """h = x + residual, y = h / rms(h) * weight and, with ``quantize`` (or ``q``
    and ``scale`` given), the normed rows in 8 bits with a scale each.

    x, residual, h, y: [rows, d] with unit stride along d (any row stride).  ``h``
    and ``y`` may be ``x`` or ``residual`` themselves.  ``want_y=False`` with
    ``quantize`` writes the 8 bits alone."""
    device, dtype, shape = x.device, x.dtype, x.shape
    code = _CODES[dtype] if dtype in _CODES else _dtype_code(dtype)
    if len(shape) != 2:
        raise ValueError(f"x must be 2-D [rows, d], got shape {tuple(shape)}")
    rows, d = shape
    ld_x = _rows(x, "x", device, dtype, shape)
    wp = _vec(weight, "weight", device, dtype, d)
    ld_r = ld_h = ld_y = d
    rp = hp = yp = qd = None
    if residual is not None:
        ld_r = _rows(residual, "residual", device, dtype, shape)
        rp = residual.data_ptr()
    if h is not None:
        ld_h = _rows(h, "h", device, dtype, shape)
        hp = h.data_ptr()
    elif residual is not None:
        h = _t.empty_like(x, memory_format=_CONTIGUOUS)
        hp = h.data_ptr()
    if y is not None:
        ld_y = _rows(y, "y", device, dtype, shape)
        yp = y.data_ptr()
    elif want_y:
        y = _t.empty_like(x, memory_format=_CONTIGUOUS)
        yp = y.data_ptr()
    if (q is None) != (scale is None):
        raise ValueError("q and scale are given together")
    if q is not None:
        qd = _int8_rows(q, scale, "q", device, shape)
    elif quantize:
        q, scale, qd = _new_int8_rows(x)
    st = _lib.twell_rmsnorm(x.data_ptr(), ld_x, rp, ld_r, wp, eps, rows, d, code, hp, ld_h, yp, ld_y, qd,
                            _raw_stream(device))
    if st:
        _check(st)
    return RmsNormOut(y, x if h is None else h, q, scale)


@functools.lru_cache(maxsize=4096)
def twell_rmsnorm_backward_workspace_size(rows: int, d: int, dtype) -> int:
    """Bytes of the gradient's workspace; 0 for sizes that it does not take."""
    if max(rows, d) > _MAX_SIZE:
        return 0
    return int(_lib.twell_rmsnorm_backward_workspace_size(rows, d, _dtype_code(dtype)))


def twell_rmsnorm_backward(dy, h, weight, eps: float = 1e-6, dh=None, dx=None, dweight=None, workspace=None):
    """Gradients of the norm from the stored h: (dx, dweight); dx [rows, d] in
    the activation dtype (the gradient of x and of the residual alike), with
    the residual stream's gradient ``dh`` added when given; dweight float32 [d]."""
    device, dtype, shape = h.device, h.dtype, h.shape
    code = _CODES[dtype] if dtype in _CODES else _dtype_code(dtype)
    if len(shape) != 2:
        raise ValueError(f"h must be 2-D [rows, d], got shape {tuple(shape)}")
    rows, d = shape
    ld_h = _rows(h, "h", device, dtype, shape)
    ld_dy = _rows(dy, "dy", device, dtype, shape)
    wp = _vec(weight, "weight", device, dtype, d)
    ld_dh = ld_dx = d
    sp = None
    if dh is not None:
        ld_dh = _rows(dh, "dh", device, dtype, shape)
        sp = dh.data_ptr()
    if dx is None:
        dx = _t.empty_like(h, memory_format=_CONTIGUOUS)
    else:
        ld_dx = _rows(dx, "dx", device, dtype, shape)
    if dweight is None:
        dweight = h.new_empty((d,), dtype=_FLOAT32)
    else:
        _vec(dweight, "dweight", device, _FLOAT32, d)
    ws = _workspace(twell_rmsnorm_backward_workspace_size(rows, d, dtype), device, workspace)
    st = _lib.twell_rmsnorm_backward(dy.data_ptr(), ld_dy, h.data_ptr(), ld_h, wp, sp, ld_dh, eps, rows, d, code,
                                     dx.data_ptr(), ld_dx, dweight.data_ptr(), ws.data_ptr(), ws.numel(),
                                     _raw_stream(device))
    if st:
        _check(st)
    return dx, dweight


def twell_quantize_rows(x, q=None, scale=None):
    """Rows of x [rows, cols] in 8 bits: (q int8 [rows, cols], scale float32 [rows]),
    x ~ q * scale[:, None]."""
    device, dtype, shape = x.device, x.dtype, x.shape
    code = _CODES[dtype] if dtype in _CODES else _dtype_code(dtype)
    if len(shape) != 2:
        raise ValueError(f"x must be 2-D [rows, cols], got shape {tuple(shape)}")
    ld_x = _rows(x, "x", device, dtype, shape)
    if (q is None) != (scale is None):
        raise ValueError("q and scale are given together")
    if q is None:
        q, scale, qd = _new_int8_rows(x)
    else:
        qd = _int8_rows(q, scale, "q", device, shape)
    st = _lib.twell_quantize_rows(x.data_ptr(), ld_x, code, qd, _raw_stream(device))
    if st:
        _check(st)
    return q, scale


@functools.lru_cache(maxsize=4096)
def twell_int8_matmul_workspace_size(M: int, N: int, K: int) -> int:
    """Bytes of the product's workspace; 0 where it needs none, and for sizes that it does not take."""
    if max(M, N, K) > _MAX_SIZE:
        return 0
    return int(_lib.twell_int8_matmul_workspace_size(M, N, K))


def twell_int8_matmul(a, a_scale, b, b_scale, row_bias=None, dtype=None, y=None, workspace=None):
    """y[m, n] = (sum_k a[m, k] b[n, k]) * a_scale[m] * b_scale[n] (+ row_bias[m])
    for int8 rows a [M, K], b [N, K] as twell_quantize_rows lays them out; y
    [M, N] in ``dtype`` (default bfloat16, or that of a given ``y``)."""
    device = a.device
    if a.dim() != 2 or b.dim() != 2:
        raise ValueError("a and b must be 2-D")
    M, K = a.shape
    N = b.shape[0]
    ad = _int8_rows(a, a_scale, "a", device, (M, K))
    bd = _int8_rows(b, b_scale, "b", device, (N, K))
    bp = None if row_bias is None else _vec(row_bias, "row_bias", device, _FLOAT32, M)
    if dtype is None:
        dtype = _BFLOAT16 if y is None else y.dtype
    code = _CODES[dtype] if dtype in _CODES else _dtype_code(dtype)
    ld_y = N
    if y is None:
        y = a_scale.new_empty((M, N), dtype=dtype)
    else:
        ld_y = _rows(y, "y", device, dtype, (M, N))
    nbytes = twell_int8_matmul_workspace_size(M, N, K)
    ws, wn = None, 0
    if nbytes:
        workspace = _workspace(nbytes, device, workspace)
        ws, wn = workspace.data_ptr(), workspace.numel()
    st = _lib.twell_int8_matmul(ad, bd, bp, code, y.data_ptr(), ld_y, ws, wn, _raw_stream(device))
    if st:
        _check(st)
    return y


# --------------------------------------------------------------------------- microscaled rows

def _launch(device, fn, *args):
    """Calls an entry point on the device's current stream, with the device current."""
    if _torch_c._cuda_getDevice() == device.index:
        st = fn(*args, _raw_stream(device))
    else:
        with _t.cuda.device(device):
            st = fn(*args, _raw_stream(device))
    if st:
        _check(st)


def _new(shape, dtype, device):
    # (0.4 us less than torch.empty)
    return _t.empty_strided(shape, (shape[1], 1), dtype=dtype, device=device)


class Mx4Rows:
    """Rows of microscaled 4-bit floats (``twell_mx4`` in include/twell.h), as
    ``twell_quantize_mx4`` lays them out: ``q`` uint8 [rows, ceil(cols / 2)] with
    16-byte aligned rows, ``scale`` uint8 [rows, ceil(cols / 32) rounded up to 16],
    ``factor`` float32 [rows] or None.  ``rows`` and ``cols`` do not change; a row
    slice of each tensor is one of fewer rows."""

    # Rows made here are one buffer (codes, scales, factors); its three tensors are
    # made when they are asked for (1.5 us each, of a decoding step's 10).
    __slots__ = ("_rows", "_cols", "_q", "_scale", "_factor", "_buf", "_has_factor")

    def __init__(self, q, scale, cols: int, factor=None):
        self._rows, self._cols = q.shape[0] if q.dim() else 0, cols
        self._q, self._scale, self._factor, self._buf = q, scale, factor, None
        self._has_factor = factor is not None

    @classmethod
    def _of(cls, buf, rows, cols, factor):
        r = cls.__new__(cls)
        r._rows, r._cols, r._buf, r._has_factor = rows, cols, buf, factor
        r._q = r._scale = r._factor = None
        return r

    @classmethod
    def empty(cls, rows: int, cols: int, device, factor: bool = False) -> "Mx4Rows":
        ld, lds = _mx4_strides(cols)
        return cls._of(_t.empty((rows * (ld + lds + (4 if factor else 0)),), dtype=_UINT8, device=device), rows, cols,
                       factor)

    def _part(self, start, width, stride):
        return self._buf.as_strided((self._rows, width), (stride, 1), start)

    @property
    def rows(self) -> int:
        return self._rows

    @property
    def cols(self) -> int:
        return self._cols

    @property
    def q(self):
        if self._q is None:
            self._q = self._part(0, (self._cols + 1) // 2, _mx4_strides(self._cols)[0])
        return self._q

    @property
    def scale(self):
        if self._scale is None:
            ld, lds = _mx4_strides(self._cols)
            self._scale = self._part(self._rows * ld, lds, lds)
        return self._scale

    @property
    def factor(self):
        if self._factor is None and self._has_factor:
            self._factor = self._buf[self._rows * sum(_mx4_strides(self._cols)):].view(_FLOAT32)
        return self._factor

    @property
    def device(self):
        return (self._q if self._buf is None else self._buf).device

    def _replace(self, **changed) -> "Mx4Rows":
        return Mx4Rows(**{**dict(q=self.q, scale=self.scale, cols=self._cols, factor=self.factor), **changed})


def _mx4_strides(cols):
    return (cols + 31) // 32 * 16, (cols + 511) // 512 * 16


def _new_mx4(x, rows, cols, factor):
    """Rows on x's device, and their descriptor."""
    ld, lds = _mx4_strides(cols)
    buf = _t.empty_strided((rows * (ld + lds + (4 if factor else 0)),), (1,), dtype=_UINT8, device=x.device)
    at = buf.data_ptr()
    return Mx4Rows._of(buf, rows, cols, factor), TwellMx4C(rows, cols, ld, at, lds, at + rows * ld,
                                                           at + rows * (ld + lds) if factor else None)


def _byte_rows(t, name, part, device, rows, cols, stride) -> int:
    """Checks codes or scales [rows, cols]; returns their row stride, or `stride` for a single row."""
    if t is None or t.dtype != _UINT8 or t.device != device or not t.is_cuda or t.shape != (rows, cols):
        _bad_rows(t, f"{name}.{part}", device, _UINT8, (rows, cols))
    across, along = t.stride()
    if along != 1 and cols > 1 and rows:
        _bad_rows(t, f"{name}.{part}", device, _UINT8, (rows, cols))
    return across if rows > 1 else stride


def _mx4_rows(r, name, device, rows, cols) -> TwellMx4C:
    """The descriptor of 4-bit rows: every row 16-byte aligned, with its last 16-byte
    chunk inside the tensor's storage."""
    if not isinstance(r, Mx4Rows):
        raise TypeError(f"{name} must be Mx4Rows, got {type(r).__name__}")
    if r._cols != cols or r._rows != rows or not 0 < cols <= _MAX_SIZE or not 0 <= rows <= _MAX_SIZE:
        raise ValueError(f"{name} must be {rows} x {cols} (with columns, each below 2^31), got {r._rows} x {r._cols}")
    wide, lds = _mx4_strides(cols)
    buf = r._buf
    if buf is not None:
        if buf.device != device:
            raise ValueError(f"{name} must be on {device}")
        at = buf.data_ptr()
        return TwellMx4C(rows, cols, wide, at, lds, at + rows * wide, at + rows * (wide + lds) if r._has_factor else None)
    q, scale, n = r._q, r._scale, (cols + 1) // 2
    ld = _byte_rows(q, name, "q", device, rows, n, wide)
    ld_scale = _byte_rows(scale, name, "scale", device, rows, lds, lds)
    fp = None if r._factor is None else _vec(r._factor, f"{name}.factor", device, _FLOAT32, rows)
    if ld % 16 or ld_scale % 16:
        raise ValueError(f"{name}: row strides {ld} and {ld_scale} are not multiples of 16 (lay rows out as "
                         "twell_quantize_mx4 does)")
    end = (n + 15) // 16 * 16
    if end != n and rows and q.storage_offset() + (rows - 1) * ld + end > q.untyped_storage().nbytes():
        raise ValueError(f"{name}: the last row's 16-byte chunks run past the tensor's storage")
    return TwellMx4C(rows, cols, ld, q.data_ptr(), ld_scale, scale.data_ptr(), fp)


def twell_quantize_mx4(x, out: Optional[Mx4Rows] = None) -> Mx4Rows:
    """Rows of x [rows, cols] in microscaled 4-bit floats."""
    device, dtype, shape = x.device, x.dtype, x.shape
    code = _CODES[dtype] if dtype in _CODES else _dtype_code(dtype)
    if len(shape) != 2:
        raise ValueError(f"x must be 2-D [rows, cols], got shape {tuple(shape)}")
    ld_x = _rows(x, "x", device, dtype, shape)
    if out is None:
        out, desc = _new_mx4(x, *shape, False)
    else:
        desc = _mx4_rows(out, "out", device, *shape)
    _launch(device, _lib.twell_quantize_mx4, x.data_ptr(), ld_x, code, desc)
    return out


def twell_dequantize_mx4(rows: Mx4Rows, dtype=None, y=None):
    """The values of 4-bit rows, [rows, cols] in ``dtype`` (default bfloat16, or
    that of a given ``y``)."""
    if not isinstance(rows, Mx4Rows):
        raise TypeError(f"rows must be Mx4Rows, got {type(rows).__name__}")
    device = rows.device
    shape = (rows._rows, rows._cols)
    desc = _mx4_rows(rows, "rows", device, *shape)
    if dtype is None:
        dtype = _BFLOAT16 if y is None else y.dtype
    code = _CODES[dtype] if dtype in _CODES else _dtype_code(dtype)
    ld_y = shape[1]
    if y is None:
        y = _new(shape, dtype, device)
    else:
        ld_y = _rows(y, "y", device, dtype, shape)
    _launch(device, _lib.twell_dequantize_mx4, desc, code, y.data_ptr(), ld_y)
    return y


class RmsNormMx4Out(NamedTuple):
    """What ``twell_rmsnorm_mx4`` wrote (None: not asked for); ``h`` is x itself without a residual."""

    y: object    # dtype [rows, d]
    h: object    # dtype [rows, d]
    q: Mx4Rows   # with a factor per row


def twell_rmsnorm_mx4(x, weight, eps: float = 1e-6, residual=None, h=None, y=None, q: Optional[Mx4Rows] = None,
                      want_y: bool = True) -> RmsNormMx4Out:
    """``twell_rmsnorm`` with the normed rows in microscaled 4-bit floats.

    x, residual, h, y: [rows, d] with unit stride along d (any row stride).  ``h``
    and ``y`` may be ``x`` or ``residual`` themselves.  ``want_y=False`` writes the
    4 bits alone."""
    device, dtype, shape = x.device, x.dtype, x.shape
    code = _CODES[dtype] if dtype in _CODES else _dtype_code(dtype)
    if len(shape) != 2:
        raise ValueError(f"x must be 2-D [rows, d], got shape {tuple(shape)}")
    rows, d = shape
    ld_x = _rows(x, "x", device, dtype, shape)
    wp = _vec(weight, "weight", device, dtype, d)
    ld_r = ld_h = ld_y = d
    rp = hp = yp = None
    if residual is not None:
        ld_r = _rows(residual, "residual", device, dtype, shape)
        rp = residual.data_ptr()
    if h is not None:
        ld_h = _rows(h, "h", device, dtype, shape)
        hp = h.data_ptr()
    elif residual is not None:
        h = _new(shape, dtype, device)
        hp = h.data_ptr()
    if y is not None:
        ld_y = _rows(y, "y", device, dtype, shape)
        yp = y.data_ptr()
    elif want_y:
        y = _new(shape, dtype, device)
        yp = y.data_ptr()
    if q is None:
        q, qd = _new_mx4(x, rows, d, True)
    else:
        qd = _mx4_rows(q, "q", device, rows, d)
    _launch(device, _lib.twell_rmsnorm_mx4, x.data_ptr(), ld_x, rp, ld_r, wp, eps, rows, d, code, hp, ld_h, yp, ld_y,
            qd)
    return RmsNormMx4Out(y, x if h is None else h, q)


@functools.lru_cache(maxsize=4096)
def twell_mx4_matmul_workspace_size(M: int, N: int, K: int) -> int:
    """Bytes of the product's workspace; 0 where it needs none, and for sizes that it does not take."""
    if max(M, N, K) > _MAX_SIZE:
        return 0
    return int(_lib.twell_mx4_matmul_workspace_size(M, N, K))


def twell_mx4_matmul(a: Mx4Rows, b: Mx4Rows, row_bias=None, dtype=None, y=None, workspace=None):
    """y[m, n] = sum_k a[m, k] b[n, k] (+ row_bias[m]) for 4-bit rows a [M, K], b [N, K]
    with their factors; y [M, N] in ``dtype`` (default bfloat16, or that of a
    given ``y``)."""
    if not isinstance(a, Mx4Rows) or not isinstance(b, Mx4Rows):
        raise TypeError(f"a and b must be Mx4Rows, got {type(a).__name__} and {type(b).__name__}")
    device = a.device
    M, N, K = a._rows, b._rows, a._cols
    ad = _mx4_rows(a, "a", device, M, K)
    bd = _mx4_rows(b, "b", device, N, K)
    bp = None if row_bias is None else _vec(row_bias, "row_bias", device, _FLOAT32, M)
    if dtype is None:
        dtype = _BFLOAT16 if y is None else y.dtype
    code = _CODES[dtype] if dtype in _CODES else _dtype_code(dtype)
    ld_y = N
    if y is None:
        y = _new((M, N), dtype, device)
    else:
        ld_y = _rows(y, "y", device, dtype, (M, N))
    nbytes = twell_mx4_matmul_workspace_size(M, N, K)
    ws, wn = None, 0
    if nbytes:
        workspace = _workspace(nbytes, device, workspace)
        ws, wn = workspace.data_ptr(), workspace.numel()
    _launch(device, _lib.twell_mx4_matmul, ad, bd, bp, code, y.data_ptr(), ld_y, ws, wn)
    return y


# --------------------------------------------------------------------------- the optimiser

@functools.lru_cache(maxsize=64)
def _adamw_struct(count: int) -> struct.Struct:
    """A list of ``count`` twell_adamw_tensor."""
    one = struct.calcsize("@q7P2if") + 4
    assert one == ctypes.sizeof(TwellAdamWTensorC)
    return struct.Struct("@" + "q7P2if4x" * count)


def _grad_list(grads):
    """(the C list, device) of gradients alone."""
    flat = []
    device = None if grads[0] is None else grads[0].device
    for g in grads:
        if g is None or g.device != device or not g.is_cuda or not g.is_contiguous():
            _need(g, "grads", device)
        dtype = g.dtype
        flat += (g.numel(), 0, 0, g.data_ptr(), 0, 0, 0, 0, 0, _CODES[dtype] if dtype in _CODES else _dtype_code(dtype), 0.0)
    return _adamw_struct(len(grads)).pack(*flat), device


def twell_grad_norm(grads, max_norm: float = float("inf"), out=None, workspace=None):
    """The norm of all gradients together and the factor that clips them to
    ``max_norm``: float32 [2], as ``twell_adamw_step`` takes it for ``clip``."""
    if not isinstance(grads, (list, tuple)):
        grads = list(grads)
    if not grads:
        raise ValueError("grads is empty")
    table, device = _grad_list(grads)
    if out is None:
        out = _t.empty((2,), dtype=_FLOAT32, device=device)
    else:
        _vec(out, "out", device, _FLOAT32, 2)
    ws = _workspace(int(_lib.twell_grad_norm_workspace_size(table, len(grads))), device, workspace)
    _launch(device, _lib.twell_grad_norm, table, len(grads), max_norm, out.data_ptr(), ws.data_ptr(), ws.numel())
    return out


_address, _nbytes = _t.Tensor.data_ptr, operator.attrgetter("nbytes")


class TwellAdamW:
    """Weights and optimiser states of ``twell_adamw_step``: tuples with an entry
    per weight tensor (``twell_adamw_tensor`` in include/twell.h), none of which
    share memory.

    m, v: float32 like the weights, or uint8 codes [numel] with ``m_scale`` and
    ``v_scale`` uint8 [ceil(numel / 32)] (None for a tensor with 32-bit states).
    master: float32 copies of bfloat16 weights, or None (for all, or for a
    tensor).  weight_decay: one number, or one per tensor.

    All of them may be assigned anew (a resumed run's states); the next step
    checks what it finds."""

    _GIVEN = frozenset(("weights", "m", "v", "m_scale", "v_scale", "master", "weight_decay"))

    def __init__(self, weights, m, v, m_scale=None, v_scale=None, master=None, weight_decay=0.0):
        self.weights, self.m, self.v = weights, m, v
        self.m_scale, self.v_scale, self.master, self.weight_decay = m_scale, v_scale, master, weight_decay
        self.validate()

    def __setattr__(self, name, value):
        if name in self._GIVEN:
            value = value if value is None or isinstance(value, (int, float)) else tuple(value)
            object.__setattr__(self, "_checked", False)
        object.__setattr__(self, name, value)

    @classmethod
    def zeros(cls, weights, bits: int = 32, master: bool = False, weight_decay=0.0) -> "TwellAdamW":
        """States before the first step, with ``bits`` 32 or 8; ``master``: keep
        float32 copies of the bfloat16 weights."""
        if bits not in (8, 32):
            raise ValueError(f"states have 8 or 32 bits, not {bits}")
        weights = tuple(weights)

        def states():
            if bits == 32:
                return [_t.zeros_like(w, dtype=_FLOAT32, memory_format=_CONTIGUOUS) for w in weights]
            return [_t.zeros((w.numel(),), dtype=_UINT8, device=w.device) for w in weights]

        def scales():
            if bits == 32:
                return None
            return [_t.zeros(((w.numel() + 31) // 32,), dtype=_UINT8, device=w.device) for w in weights]

        copies = [w.detach().float() if w.dtype == _BFLOAT16 else None for w in weights] if master else None
        return cls(weights, states(), states(), scales(), scales(), copies, weight_decay)

    def validate(self) -> None:
        """Check every buffer before its pointers reach the library."""
        weights = self.weights
        if not weights:
            raise ValueError("no weights")
        n, device = len(weights), weights[0].device
        lists = {"weights": weights}
        for name in ("master", "m", "v", "m_scale", "v_scale"):
            given = getattr(self, name)
            lists[name] = (None,) * n if given is None else given
        decay = self.weight_decay
        decay = (float(decay),) * n if isinstance(decay, (int, float)) else tuple(float(d) for d in decay)
        for name, entries in (*lists.items(), ("weight_decay", decay)):
            if len(entries) != n:
                raise ValueError(f"{name}: {len(entries)} entries, {n} weights")

        def need(t, name, i, dtype, shape):
            if (t is None or t.dtype != dtype or t.shape != shape or t.device != device or not t.is_cuda
                    or not t.is_contiguous()):
                _need(t, f"{name}[{i}]", device, dtype, shape)

        for i, (w, x, m, v, ms, vs) in enumerate(zip(*lists.values())):
            dtype, shape = w.dtype, w.shape
            need(w, "weights", i, dtype, shape)
            if dtype not in _CODES:
                _dtype_code(dtype)
            if (ms is None) != (vs is None):
                raise ValueError(f"m_scale[{i}] and v_scale[{i}] go together")
            if ms is None:
                need(m, "m", i, _FLOAT32, shape)
                need(v, "v", i, _FLOAT32, shape)
            else:
                codes = (w.numel(),)
                blocks = ((codes[0] + 31) // 32,)
                need(m, "m", i, _UINT8, codes)
                need(ms, "m_scale", i, _UINT8, blocks)
                need(v, "v", i, _UINT8, codes)
                need(vs, "v_scale", i, _UINT8, blocks)
            if x is not None:
                if dtype == _FLOAT32:
                    raise ValueError(f"master[{i}]: float32 weights have no float32 copy")
                need(x, "master", i, _FLOAT32, shape)
        # a step writes all of them, in no order between tensors
        names = [(name, i) for name, entries in lists.items() for i, t in enumerate(entries) if t is not None]
        others = [t for entries in list(lists.values())[1:] for t in entries if t is not None]
        all_ = [*weights, *others]
        at, sizes = list(map(_address, all_)), list(map(_nbytes, all_))
        spans = sorted((start, start + size, name) for start, size, name in zip(at, sizes, names) if size)
        for t, size, (name, i) in zip(all_, sizes, names):
            if t.untyped_storage().nbytes() < size:
                raise ValueError(f"{name}[{i}]: its storage has been given back")
        for (_, end, one), (start, _, two) in zip(spans, spans[1:]):
            if start < end:
                raise ValueError(f"{one[0]}[{one[1]}] and {two[0]}[{two[1]}] share memory")
        for name, entries in lists.items():
            setattr(self, name, entries)
        self.weight_decay, self.device = decay, device
        self._versioned = [*weights, *(x for x in lists["master"] if x is not None)]
        self._views = [None if w.dim() == 1 else w.shape for w in weights] * 2  # of the states' values
        self._scales = {None if ms is None else True for ms in lists["m_scale"]}
        # where the written memory begins and ends, in turn
        self._bounds = [end for span in spans for end in span[:2]] + [1 << 64]
        self._shapes, self._dtypes = [w.shape for w in weights], [w.dtype for w in weights]
        # A buffer of the same address and bytes is the one checked here; weights are given
        # other storage from outside now and then.
        self._others, self._others_at, self._weights_at = others, (at[n:], sizes[n:]), (at[:n], sizes[:n])
        # the C list but for the gradients: all that reading the states takes
        where = {name: [0] * n for name in lists}
        for (name, i), start in zip(names, at):
            where[name][i] = start
        self._fields = [0] * (11 * n)
        self._fields[::11] = [w.numel() for w in weights]
        for k, name in ((1, "weights"), (2, "master"), (4, "m"), (5, "v"), (6, "m_scale"), (7, "v_scale")):
            self._fields[k::11] = where[name]
        self._fields[8::11] = [_CODES[w.dtype] for w in weights]
        self._fields[10::11] = decay
        self._states = _adamw_struct(n).pack(*self._fields)
        self._checked = True

    def _check(self) -> None:
        """validate() anew where a buffer is not the one that it has seen."""
        if not self._checked or (list(map(_address, self._others)), list(map(_nbytes, self._others))) != self._others_at:
            self.validate()

    def c_list(self, grads) -> bytes:
        """The C list with this step's gradients."""
        self._check()
        weights, device = self.weights, self.device
        if (list(map(_address, weights)), list(map(_nbytes, weights))) != self._weights_at:
            for w, dtype, shape in zip(weights, self._dtypes, self._shapes):
                _need(w, "weights", device, dtype, shape)
            self.validate()
        flat, bounds, find = self._fields.copy(), self._bounds, bisect.bisect_right
        at, codes = [], []
        for w, dtype, shape, n, g in zip(weights, self._dtypes, self._shapes, flat[::11], grads):
            if g is None or g.shape != shape or g.device != device or not g.is_contiguous():
                _need(g, "grads", device, None, shape)
            if w.dtype != dtype or not w.is_contiguous():
                _need(w, "weights", device, dtype, shape)
            kind, start = g.dtype, g.data_ptr()
            code = _CODES[kind] if kind in _CODES else _dtype_code(kind)
            i = find(bounds, start)
            if (i & 1 or bounds[i] < start + n * _SIZES[code]) and n:  # inside a buffer, or up into the next one
                raise ValueError(f"grads[{len(at)}] and a buffer that the step writes share memory")
            at.append(start)
            codes.append(code)
        flat[3::11], flat[9::11] = at, codes
        return _adamw_struct(len(weights)).pack(*flat)

    def c_states(self) -> bytes:
        """The C list for reading the states."""
        self._check()
        return self._states


def twell_adamw_step(opt: TwellAdamW, grads, lr, step, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
                     clip=None, seed: int = 0) -> None:
    """One AdamW step over all of ``opt``'s tensors, in place, with ``grads``
    (float32 or bfloat16) like the weights, none of them in memory that it writes.

    ``step`` counts from 1; it or ``lr`` may be a tensor of one element on the GPU
    (int64, float32), read when the step runs.  ``clip``: what ``twell_grad_norm``
    returned (a factor that is not finite leaves the step out).  ``seed``: of the
    random roundings of 8-bit states and of bfloat16 weights without a copy.

    Autograd counts the step as a change in place, as torch's optimisers do: a
    backward through a graph that saved a weight before it raises."""
    if not isinstance(grads, (list, tuple)):
        grads = list(grads)
    if len(grads) != len(opt.weights):
        raise ValueError(f"{len(grads)} gradients, {len(opt.weights)} weights")
    table = opt.c_list(grads)
    device = opt.device
    lp = sp = cp = None
    if isinstance(lr, _t.Tensor):
        lp, lr = _one(lr, "lr", device, _FLOAT32), 0.0
    if isinstance(step, _t.Tensor):
        sp, step = _one(step, "step", device, _INT64), 1
    elif not 1 <= step < 1 << 63:
        raise ValueError(f"steps count from 1, got {step}")
    if clip is not None:
        cp = _vec(clip, "clip", device, _FLOAT32, 2)
    args = TwellAdamWC(lr, beta1, beta2, eps, step, seed & 0xFFFFFFFFFFFFFFFF, lp, sp)
    _launch(device, _lib.twell_adamw_step, table, len(grads), args, cp)
    _t.autograd.graph.increment_version(opt._versioned)


def _one(t, name, device, dtype) -> int:
    if t.numel() != 1:
        raise ValueError(f"{name} must have one element, got {t.numel()}")
    _need(t, name, device, dtype)
    return t.data_ptr()


def twell_adamw_states(opt: TwellAdamW, dtype=None):
    """The values of ``opt``'s 8-bit states, (m, v): lists of tensors like the weights
    in ``dtype`` (default bfloat16, which holds them exactly)."""
    dtype = _BFLOAT16 if dtype is None else dtype
    code = _dtype_code(dtype)
    table = opt.c_states()
    if None in opt._scales:
        raise ValueError("states of 32 bits need no reading")
    # one buffer for all: two calls for the 2 n tensors
    n = len(opt.weights)
    sizes = opt._fields[::11] * 2
    whole = _t.empty((sum(sizes),), dtype=dtype, device=opt.device)
    size, base = _SIZES[code], whole.data_ptr()
    at = [base + size * k for k in itertools.accumulate(sizes, initial=0)]
    parts = whole.split_with_sizes(sizes)
    pointers = struct.Struct(f"@{n}P").pack
    _launch(opt.device, _lib.twell_adamw_states, table, n, code, pointers(*at[:n]), pointers(*at[n:-1]))
    values = [t if shape is None else t.view(shape) for t, shape in zip(parts, opt._views)]
    return values[:n], values[n:]


def twell_stream_probe(src, dst, mode: int) -> None:
    """Streaming HBM probe on the current stream: mode 0 reads src (dst is a
    device sink of at least 4 bytes), mode 1 copies src into dst."""
    device = src.device
    _need(src, "src", device)
    _need(dst, "dst", device)
    nbytes = src.numel() * src.element_size()
    if mode == 1 and dst.numel() * dst.element_size() < nbytes:
        raise ValueError("dst is smaller than src")
    if mode == 0 and dst.numel() * dst.element_size() < 4:
        raise ValueError("the sink needs 4 bytes")
    _check(_lib.twell_stream_probe(_ptr(src), _ptr(dst), nbytes, mode, _stream(device)))


def twell_mfma_probe(sink, iters: int, blocks: int) -> float:
    """Matrix-core probe on the current stream; returns the flops it performs
    (sink: a device tensor of at least 4 bytes)."""
    _need(sink, "sink", sink.device)
    if sink.numel() * sink.element_size() < 4:
        raise ValueError("the sink needs 4 bytes")
    _check(_lib.twell_mfma_probe(_ptr(sink), iters, blocks, _stream(sink.device)))
    return 2.0 * 32 * 32 * 16 * 8 * iters * 8 * blocks
