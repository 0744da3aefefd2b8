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

_TYPE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_HALF = {torch.float16: 1, torch.bfloat16: 2}
_Tensor, _empty = torch.Tensor, torch.empty
_F32, _I32, _I8, _U8 = torch.float32, torch.int32, torch.int8, torch.uint8

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


def grouped_config_count() -> int:
    """Number of kernels the grouped and MXFP4 products choose from."""
    return int(load_library().lpgemm_grouped_config_count())


def force_grouped_config(config: int) -> int:
    """Pin kernel `config` for later grouped and MXFP4 products in this process
    (-1: by size); returns the previous setting."""
    return int(load_library().lpgemm_force_grouped_config(int(config)))


GROUPED_KINDS = {"f16": 2, "i8": 3, "mxfp4": 6}


def grouped_auto_config(kind: str, rows: int, groups: int, N: int, K: int, cu_count: int) -> int:
    """The kernel a grouped product of `kind` ("i8", "f16" or "mxfp4") takes on
    `cu_count` compute units (-1: nothing is launched or out of range)."""
    f = load_library().lpgemm_grouped_auto_config
    f.argtypes = [_int, _i64, _i64, _i64, _i64, _int]
    return int(f(GROUPED_KINDS[kind], rows, groups, N, K, cu_count))


def _stream_of(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# torch's own accessor of the current stream's handle, without a Stream object
_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _stream_of)


def _call(name: str, dev, *args) -> None:
    """The entry point `name` on the current stream of `dev`."""
    f = _functions.get(name) or _function(name)
    index = dev.index
    if index == torch.cuda.current_device():
        status = f(*args, _stream(index))
    else:
        with torch.cuda.device(dev):
            status = f(*args, _stream(index))
    if status:
        raise LpgemmError(status, name)


def _refuse(t, name, dtypes, shape=None, dev=None, dims=None):
    """Says what is wrong with a tensor that failed a check."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if dims is not None and t.dim() != dims:
        raise ValueError(f"{name} must be {dims}-D, got shape {tuple(t.shape)}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU device")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} must be on {dev}, as the other tensors are")
    raise ValueError(f"{name} must be contiguous")


def _full(t, name, dtype, shape, dev):
    """A contiguous tensor of that type and shape on `dev`."""
    if not isinstance(t, _Tensor) or t.dtype is not dtype or t.shape != shape or t.device != dev \
            or not t.is_contiguous():
        _refuse(t, name, (dtype,), shape, dev)


def _operand(t, name, dtype, dims):
    """A contiguous GPU tensor of that type."""
    if not isinstance(t, _Tensor) or t.dtype is not dtype or t.dim() != dims or not t.is_cuda \
            or not t.is_contiguous():
        _refuse(t, name, (dtype,), dims=dims)


def _rows(t, name, dtypes):
    """A matrix whose rows are contiguous: (rows, columns, row stride), the
    stride being the row's length where no element uses it."""
    if not isinstance(t, _Tensor) or t.dtype not in dtypes or t.dim() != 2 or not t.is_cuda:
        _refuse(t, name, dtypes, dims=2)
    M, K = t.shape
    if M == 0 or K == 0:
        return M, K, K
    stride, along = t.stride()
    if along != 1 and K > 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    return M, K, stride if M > 1 else K


def _out(out, name, shape, dtype, dev):
    if out is None:
        return _empty(*shape, dtype=dtype, device=dev)   # (a tuple takes torch a third longer)
    _full(out, name, dtype, shape, dev)
    return out


def _row_stride(t, name, x):
    """The row stride of a matrix that must go with x."""
    M, K, stride = _rows(t, name, (x.dtype,))
    if t.shape != x.shape or t.device != x.device:
        raise ValueError(f"{name} must have x's shape {tuple(x.shape)} and be on {x.device}")
    return stride


def add_rmsnorm_quantize(x, weight, eps: float, residual=None, residual_out=None, q_out=None, scale_out=None):
    """Residual addition, RMSNorm and int8 rows: returns (q int8 M x K, scale
    fp32 M, h) with h = x + residual in x's type (without a residual, h is x)
    and q * scale[:, None] the normalised row times `weight`.

    x, residual: M x K fp16 or bf16 whose rows are contiguous and whose row
    stride is a multiple of 8; weight: K values of the same type.  h goes to
    `residual_out` (M x K, may be x or residual itself) or a new tensor.  A
    row with a non-finite value gets scale NaN and codes 0."""
    M, K, stride = _rows(x, "x", _HALF)
    dev, dtype = x.device, x.dtype
    _full(weight, "weight", dtype, (K,), dev)
    h, r_ptr, r_stride, h_ptr, h_stride = residual_out, None, 0, None, 0
    if residual is not None:
        r_stride = _row_stride(residual, "residual", x)
        r_ptr = residual.data_ptr()
        if h is None:
            h = _empty(M, K, dtype=dtype, device=dev)
    if h is None:
        h = x
    else:
        h_stride = _row_stride(h, "residual_out", x)
        h_ptr = h.data_ptr()
    q = _out(q_out, "q_out", (M, K), _I8, dev)
    scale = _out(scale_out, "scale_out", (M,), _F32, dev)
    _call("lpgemm_add_rmsnorm_quantize", dev, M, K, _HALF[dtype], x.data_ptr(), stride, r_ptr, r_stride,
          weight.data_ptr(), eps, h_ptr, h_stride, q.data_ptr(), scale.data_ptr())
    return q, scale, h


def silu_mul_quantize(x, q_out=None, scale_out=None):
    """silu(gate) * up with int8 rows: x is M x 2K fp16 or bf16, a row's K gate
    values before its K up values (contiguous rows, a row stride that is a
    multiple of 8); returns (q int8 M x K, scale fp32 M)."""
    M, K2, stride = _rows(x, "x", _HALF)
    if K2 % 2:
        raise ValueError(f"x must have an even number of columns, got {K2}")
    K, dev = K2 // 2, x.device
    q = _out(q_out, "q_out", (M, K), _I8, dev)
    scale = _out(scale_out, "scale_out", (M,), _F32, dev)
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
    rows, K, stride = _rows(x, "x", _HALF)
    dev = x.device
    codes = _out(codes_out, "codes_out", (rows, K // 2), _U8, dev)
    scales = _out(scales_out, "scales_out", (rows, mxfp4_scale_stride(K)), _U8, dev)
    _call("lpgemm_quantize_mxfp4", dev, rows, K, _HALF[x.dtype], x.data_ptr(), stride, codes.data_ptr(),
          scales.data_ptr())
    return codes, scales


def _mxfp4_operand(codes, scales, name, dims):
    _operand(codes, name, _U8, dims)
    *rows, half = codes.shape
    K = 2 * half
    _full(scales, name + "_scale", _U8, (*rows, mxfp4_scale_stride(K)), codes.device)
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


def _routing(a, b, offsets, row_index):
    """Checks the groups of a product (a and b are checked on their own):
    (rows of C, rows of a, groups, N, row_index's address)."""
    dev = a.device
    groups, N, width = b.shape
    a_rows, own = a.shape
    if own != width:
        raise ValueError(f"K mismatch: a {tuple(a.shape)}, b {tuple(b.shape)}")
    if b.device != dev:
        raise ValueError("all tensors must be on the same device")
    _full(offsets, "offsets", _I32, (groups + 1,), dev)
    if row_index is None:
        return a_rows, a_rows, groups, N, None
    _operand(row_index, "row_index", _I32, 1)
    if row_index.device != dev:
        raise ValueError("all tensors must be on the same device")
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
    _operand(a, "a", _I8, 2)
    _operand(b_t, "b_t", _I8, 3)
    rows, a_rows, groups, N, index = _routing(a, b_t, offsets, row_index)
    dev = a.device
    _full(row_scale, "row_scale", _F32, (a_rows,), dev)
    _full(col_scale, "col_scale", _F32, (groups, N), dev)
    out = _out(out, "out", (rows, N), _out_dtype(out_dtype), dev)
    _call("lpgemm_i8_dequant_grouped", dev, rows, groups, N, a.shape[1], a_rows, a.data_ptr(), b_t.data_ptr(),
          offsets.data_ptr(), index, row_scale.data_ptr(), col_scale.data_ptr(), _TYPE[out_dtype], out.data_ptr())
    return out


def gemm_f16_grouped(a, b_t, offsets, row_index: Optional[torch.Tensor] = None, out_dtype=torch.float32, out=None):
    """gemm_i8_dequant_grouped for fp16 operands, summed in fp32, without
    scales: C[i] = a[row_index[i]] . b_t[g]."""
    _operand(a, "a", torch.float16, 2)
    _operand(b_t, "b_t", torch.float16, 3)
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
