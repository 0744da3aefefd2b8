"""Binding of the expert-layer operators declared in include/lpgemm_moe.h.

As in _binding.py, every function checks its tensors (type, shape, strides,
device), allocates with torch what is not passed in, and calls the library's
entry point on the current torch stream of the tensors' device.  The checks
are kept short: at one token the kernels take a few microseconds, and so must
the call.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from ._binding import LpgemmError, load_library

_i64, _p, _int, _f32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_float

MAX_GROUPS = 65536
MAX_K_MXFP4 = 1048576

_TYPE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_HALF = {torch.float16: 1, torch.bfloat16: 2}

_SIGNATURES = {
    "lpgemm_add_rmsnorm_quantize": [_i64, _i64, _int, _p, _i64, _p, _i64, _p, _f32, _p, _i64, _p, _p, _p],
    "lpgemm_silu_mul_quantize": [_i64, _i64, _int, _p, _i64, _p, _p, _p],
    "lpgemm_quantize_mxfp4": [_i64, _i64, _int, _p, _i64, _p, _p, _p],
    "lpgemm_dequantize_mxfp4": [_i64, _i64, _p, _p, _int, _p, _p],
    "lpgemm_mxfp4": [_i64, _i64, _i64, _p, _p, _p, _p, _int, _p, _p],
    "lpgemm_i8_dequant_grouped": [_i64, _i64, _i64, _i64, _i64, _p, _p, _p, _p, _p, _p, _int, _p, _p],
    "lpgemm_f16_grouped": [_i64, _i64, _i64, _i64, _i64, _p, _p, _p, _p, _int, _p, _p],
    "lpgemm_mxfp4_grouped": [_i64, _i64, _i64, _i64, _i64, _p, _p, _p, _p, _p, _p, _int, _p, _p],
}
_functions: dict = {}


def _function(name: str):
    f = _functions.get(name)
    if f is None:
        f = getattr(load_library(), name)
        f.argtypes = _SIGNATURES[name]
        f.restype = ctypes.c_int
        _functions[name] = f
    return f


def _call(name: str, dev, *args) -> None:
    """The entry point `name` on the current stream of `dev`."""
    f = _functions.get(name) or _function(name)
    index = dev.index
    if index == torch.cuda.current_device():
        status = f(*args, torch.cuda.current_stream(dev).cuda_stream)
    else:
        with torch.cuda.device(dev):
            status = f(*args, torch.cuda.current_stream(dev).cuda_stream)
    if status:
        raise LpgemmError(status, name)


def _tensor(t, name, dtypes, dims):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.dim() != dims:
        raise ValueError(f"{name} must be {dims}-D, got shape {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU device")


def _full(t, name, dtypes, shape, dev):
    """A contiguous tensor of that shape."""
    _tensor(t, name, dtypes, len(shape))
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _rows(t, name, dtypes):
    """A matrix whose rows are contiguous; returns its row stride (a stride
    that no element uses counts as the row's length)."""
    _tensor(t, name, dtypes, 2)
    M, K = t.shape
    if K > 1 and t.stride(1) != 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    return t.stride(0) if M > 1 and K else K


def _out(out, name, shape, dtype, dev):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _full(out, name, (dtype,), torch.Size(shape), dev)
    return out


def add_rmsnorm_quantize(x, weight, eps: float, residual=None, residual_out=None, q_out=None, scale_out=None):
    """Residual addition, RMSNorm and int8 rows: returns (q int8 M x K, scale
    fp32 M, h) with h = x + residual in x's type (without a residual, h is x)
    and q * scale[:, None] the normalised row times `weight`.

    x, residual: M x K fp16 or bf16 whose rows are contiguous and whose row
    stride is a multiple of 8; weight: K values of the same type.  h goes to
    `residual_out` (M x K, may be x or residual itself) or a new tensor.  A
    row with a non-finite value gets scale NaN and codes 0."""
    stride = _rows(x, "x", _HALF)
    M, K = x.shape
    dev, dtype = x.device, x.dtype
    _full(weight, "weight", (dtype,), torch.Size((K,)), dev)
    h, r_ptr, r_stride, h_ptr, h_stride = x, None, 0, None, 0
    if residual is not None:
        r_stride = _rows(residual, "residual", (dtype,))
        if residual.shape != x.shape or residual.device != dev:
            raise ValueError(f"residual must have x's shape {(M, K)} and device")
        r_ptr = residual.data_ptr()
        h = torch.empty((M, K), dtype=dtype, device=dev) if residual_out is None else residual_out
    elif residual_out is not None:
        h = residual_out
    if h is not x or residual is not None:
        h_stride = _rows(h, "residual_out", (dtype,))
        if h.shape != x.shape or h.device != dev:
            raise ValueError(f"residual_out must have x's shape {(M, K)} and device")
        h_ptr = h.data_ptr()
    q = _out(q_out, "q_out", (M, K), torch.int8, dev)
    scale = _out(scale_out, "scale_out", (M,), torch.float32, dev)
    _call("lpgemm_add_rmsnorm_quantize", dev, M, K, _HALF[dtype], x.data_ptr(), stride, r_ptr, r_stride,
          weight.data_ptr(), eps, h_ptr, h_stride, q.data_ptr(), scale.data_ptr())
    return q, scale, h


def silu_mul_quantize(x, q_out=None, scale_out=None):
    """silu(gate) * up with int8 rows: x is M x 2K fp16 or bf16, a row's K gate
    values before its K up values (contiguous rows, a row stride that is a
    multiple of 8); returns (q int8 M x K, scale fp32 M)."""
    stride = _rows(x, "x", _HALF)
    M, K2 = x.shape
    if K2 % 2:
        raise ValueError(f"x must have an even number of columns, got {K2}")
    K, dev = K2 // 2, x.device
    q = _out(q_out, "q_out", (M, K), torch.int8, dev)
    scale = _out(scale_out, "scale_out", (M,), torch.float32, dev)
    _call("lpgemm_silu_mul_quantize", dev, M, K, _HALF[x.dtype], x.data_ptr(), stride, q.data_ptr(), scale.data_ptr())
    return q, scale


def mxfp4_scale_stride(K: int) -> int:
    """Bytes per row of an MXFP4 operand's scales: one per 32 values of k,
    padded to a multiple of 16 (no padding where K is a multiple of 512)."""
    return (K // 32 + 15) // 16 * 16


def quantize_mxfp4(x, codes_out=None, scales_out=None):
    """MXFP4 codes (rows x K/2 uint8, the even k in the low nibble) and scales
    (rows x mxfp4_scale_stride(K) uint8, E8M0) of x, rows x K fp16 or bf16
    with contiguous rows and a row stride that is a multiple of 8; K a
    multiple of 32.  Weights of several experts: quantise them as one matrix
    of groups * N rows and reshape the results."""
    stride = _rows(x, "x", _HALF)
    rows, K = x.shape
    dev = x.device
    codes = _out(codes_out, "codes_out", (rows, K // 2), torch.uint8, dev)
    scales = _out(scales_out, "scales_out", (rows, mxfp4_scale_stride(K)), torch.uint8, dev)
    _call("lpgemm_quantize_mxfp4", dev, rows, K, _HALF[x.dtype], x.data_ptr(), stride, codes.data_ptr(),
          scales.data_ptr())
    return codes, scales


_U8 = (torch.uint8,)


def _mxfp4_operand(codes, scales, name, dims):
    _tensor(codes, name, _U8, dims)
    if not codes.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    K = 2 * codes.shape[-1]
    _full(scales, name + "_scale", _U8, torch.Size((*codes.shape[:-1], mxfp4_scale_stride(K))), codes.device)
    return K


def dequantize_mxfp4(codes, scales, out_dtype=torch.float32, out=None):
    """The values that MXFP4 codes and scales stand for, rows x K in
    `out_dtype` (fp32, fp16 or bf16)."""
    K = _mxfp4_operand(codes, scales, "codes", 2)
    rows, dev = codes.shape[0], codes.device
    out = _out(out, "out", (rows, K), _out_dtype(out_dtype), dev)
    _call("lpgemm_dequantize_mxfp4", dev, rows, K, codes.data_ptr(), scales.data_ptr(), _TYPE[out_dtype],
          out.data_ptr())
    return out


def _out_dtype(dtype):
    if dtype not in _TYPE:
        raise TypeError(f"out_dtype must be torch.float32, torch.float16 or torch.bfloat16, got {dtype}")
    return dtype


def gemm_mxfp4(a, a_scale, b, b_scale, out_dtype=torch.float32, out=None):
    """C = A . B for MXFP4 operands: a (M x K/2 codes) and b (N x K/2 codes,
    K-contiguous) with their scales; C is M x N in `out_dtype`."""
    K = _mxfp4_operand(a, a_scale, "a", 2)
    if _mxfp4_operand(b, b_scale, "b", 2) != K:
        raise ValueError(f"K mismatch: a {tuple(a.shape)}, b {tuple(b.shape)}")
    M, N, dev = a.shape[0], b.shape[0], a.device
    if b.device != dev:
        raise ValueError("all tensors must be on the same device")
    out = _out(out, "out", (M, N), _out_dtype(out_dtype), dev)
    _call("lpgemm_mxfp4", dev, M, N, K, a.data_ptr(), a_scale.data_ptr(), b.data_ptr(), b_scale.data_ptr(),
          _TYPE[out_dtype], out.data_ptr())
    return out


_I32 = (torch.int32,)


def _routing(a, b, offsets, row_index):
    """Checks the groups of a product: (rows of C, rows of a, groups, N)."""
    dev = a.device
    groups, N, width = b.shape
    if a.shape[1] != width:
        raise ValueError(f"K mismatch: a {tuple(a.shape)}, b_t {tuple(b.shape)}")
    if not a.is_contiguous() or not b.is_contiguous():
        raise ValueError("a and b_t must be contiguous")
    if b.device != dev:
        raise ValueError("all tensors must be on the same device")
    _full(offsets, "offsets", _I32, torch.Size((groups + 1,)), dev)
    a_rows = a.shape[0]
    if row_index is None:
        return a_rows, a_rows, groups, N, None
    _tensor(row_index, "row_index", _I32, 1)
    if row_index.device != dev or not row_index.is_contiguous():
        raise ValueError(f"row_index must be a contiguous vector on {dev}")
    return row_index.shape[0], a_rows, groups, N, row_index.data_ptr()


def gemm_i8_dequant_grouped(a, b_t, offsets, row_scale, col_scale, row_index: Optional[torch.Tensor] = None,
                            out_dtype=torch.float32, out=None):
    """Rows sorted by expert times that expert's int8 weights:
    C[i] = (float)(a[row_index[i]] . b_t[g]) * row_scale[row_index[i]] *
    col_scale[g] for the rows i of group g, offsets[g] <= i < offsets[g + 1].

    a: tokens x K int8; b_t: groups x N x K int8; offsets: groups + 1 int32;
    row_index: int32, one per row of C (None: row i is a's row i); row_scale:
    fp32, one per row of a; col_scale: groups x N fp32.  offsets and row_index
    are read on the device.  Rows outside every group are not written."""
    _tensor(a, "a", (torch.int8,), 2)
    _tensor(b_t, "b_t", (torch.int8,), 3)
    rows, a_rows, groups, N, index = _routing(a, b_t, offsets, row_index)
    dev = a.device
    _full(row_scale, "row_scale", (torch.float32,), torch.Size((a_rows,)), dev)
    _full(col_scale, "col_scale", (torch.float32,), torch.Size((groups, N)), dev)
    out = _out(out, "out", (rows, N), _out_dtype(out_dtype), dev)
    _call("lpgemm_i8_dequant_grouped", dev, rows, groups, N, a.shape[1], a_rows, a.data_ptr(), b_t.data_ptr(),
          offsets.data_ptr(), index, row_scale.data_ptr(), col_scale.data_ptr(), _TYPE[out_dtype], out.data_ptr())
    return out


def gemm_f16_grouped(a, b_t, offsets, row_index: Optional[torch.Tensor] = None, out_dtype=torch.float32, out=None):
    """gemm_i8_dequant_grouped for fp16 operands, summed in fp32, without
    scales: C[i] = a[row_index[i]] . b_t[g]."""
    _tensor(a, "a", (torch.float16,), 2)
    _tensor(b_t, "b_t", (torch.float16,), 3)
    rows, a_rows, groups, N, index = _routing(a, b_t, offsets, row_index)
    dev = a.device
    out = _out(out, "out", (rows, N), _out_dtype(out_dtype), dev)
    _call("lpgemm_f16_grouped", dev, rows, groups, N, a.shape[1], a_rows, a.data_ptr(), b_t.data_ptr(),
          offsets.data_ptr(), index, _TYPE[out_dtype], out.data_ptr())
    return out


def gemm_mxfp4_grouped(a, a_scale, b, b_scale, offsets, row_index: Optional[torch.Tensor] = None,
                       out_dtype=torch.float32, out=None):
    """gemm_i8_dequant_grouped for MXFP4 operands: a (tokens x K/2 codes) and b
    (groups x N x K/2 codes), each with its scales."""
    K = _mxfp4_operand(a, a_scale, "a", 2)
    _mxfp4_operand(b, b_scale, "b", 3)
    rows, a_rows, groups, N, index = _routing(a, b, offsets, row_index)
    dev = a.device
    out = _out(out, "out", (rows, N), _out_dtype(out_dtype), dev)
    _call("lpgemm_mxfp4_grouped", dev, rows, groups, N, K, a_rows, a.data_ptr(), a_scale.data_ptr(), b.data_ptr(),
          b_scale.data_ptr(), offsets.data_ptr(), index, _TYPE[out_dtype], out.data_ptr())
    return out
