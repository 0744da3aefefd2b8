"""Binding of the operators declared in include/lpgemm_ffn.h: 4-bit weights
with group scales, and the gated feed-forward block with its gradients.

As in _moe.py, every function checks its tensors (type, shape, strides,
device), allocates with torch what is not passed in, and calls the library's
entry point on the current torch stream of the tensors' device.  None of them is
part of torch's automatic differentiation: what they return carries no gradient,
whatever their inputs require.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _moe
from ._binding import load_library
from ._moe import _F32, _HALF, _TYPE, _U8, _call, _empty, _f32, _full, _i64, _int, _operand, _out, _out_dtype, _p, _refuse, _rows  # noqa: F401

GROUPS = (32, 64, 128, 256)
W4_SHORT_M = 4          # up to this many rows the products with 4-bit weights need no workspace
_ACTIVATION = {"silu": 0, "gelu": 1}

_SIGNATURES = {
    "lpgemm_quantize_w4": [_i64, _i64, _i64, _int, _p, _i64, _p, _p, _p, _p],
    "lpgemm_dequantize_w4": [_i64, _i64, _i64, _int, _p, _p, _p, _int, _p, _p],
    "lpgemm_w4": [_i64, _i64, _i64, _i64, _int, _p, _i64, _p, _p, _p, _int, _p, _p, _i64, _p],
    "lpgemm_gated_w4": [_i64, _i64, _i64, _i64, _int, _int, _p, _i64, _p, _p, _p, _int, _p, _p, _i64, _p],
    "lpgemm_gated_ffn": [_i64, _i64, _i64, _int, _int, _p, _i64, _p, _p, _p, _p, _p, _i64, _p],
    "lpgemm_gated_ffn_backward": [_i64, _i64, _i64, _int, _int, _p, _i64, _p, _i64, _p, _p, _p, _int, _p, _p, _p,
                                  _p, _i64, _p],
}
_moe._SIGNATURES_ELSEWHERE.update(_SIGNATURES)

_sizes: dict = {}


def _size(name: str, *args) -> int:
    f = _sizes.get(name)
    if f is None:
        f = getattr(load_library(), name)
        f.argtypes = [_i64] * 4 + [_int] if name == "lpgemm_w4_workspace" else [_i64] * 3
        f.restype = _i64
        _sizes[name] = f
    return f(*args)


def _size_on(dev, name: str, *args) -> int:
    """A workspace's size on that device; 0 for sizes the call itself will refuse."""
    if dev.index == torch.cuda.current_device():
        return max(_size(name, *args), 0)
    with torch.cuda.device(dev):
        return max(_size(name, *args), 0)


def _activation(name) -> int:
    a = _ACTIVATION.get(name)
    if a is None:
        raise ValueError(f"activation must be 'silu' or 'gelu', got {name!r}")
    return a


def ffn_config_count() -> int:
    """Number of kernels force_ffn_config can pin."""
    return int(load_library().lpgemm_ffn_config_count())


def force_ffn_config(config: int) -> int:
    """Pin kernel `config` for later calls of these operators in this process
    (-1: by size); returns the previous setting."""
    return int(load_library().lpgemm_force_ffn_config(int(config)))


def quantize_w4(w, group_size: int = 128, zeros: bool = False, codes_out=None, scales_out=None, zeros_out=None):
    """4-bit codes of weights w, N x K fp16 or bf16 (contiguous rows, a row
    stride that is a multiple of 8), in groups of `group_size` (32, 64, 128 or
    256, a divisor of K) along k: returns (codes, scales), with `zeros` (codes,
    scales, zeros).  codes: N x K/2 uint8, two's complement, the even k in the
    low nibble; scales and zeros: N x K/group_size of w's type.  A weight is
    (code - zero) * scale.  Without zeros the scale is the group's largest
    magnitude over 7; with them the group's range, extended to 0, over 15."""
    N, K, stride = _rows(w, "w", _HALF)
    if group_size not in GROUPS or K % group_size:
        raise ValueError(f"group_size must be one of {GROUPS} and divide K = {K}, got {group_size}")
    dev, t, shape = w.device, w.dtype, (N, K // group_size)
    if zeros_out is not None and not zeros:
        raise ValueError("zeros_out goes with zeros=True")
    codes = _out(codes_out, "codes_out", (N, K // 2), _U8, dev)
    scales = _out(scales_out, "scales_out", shape, t, dev)
    zero = _out(zeros_out, "zeros_out", shape, t, dev) if zeros else None
    _call("lpgemm_quantize_w4", dev, N, K, group_size, _HALF[t], w.data_ptr(), stride, codes.data_ptr(),
          scales.data_ptr(), zero.data_ptr() if zeros else None)
    return (codes, scales, zero) if zeros else (codes, scales)


def _w4(codes, scales, zeros):
    """Checks 4-bit weights: (N, K, group size, address of zeros)."""
    _operand(codes, "codes", _U8, 2)
    N, half = codes.shape
    if not isinstance(scales, torch.Tensor) or scales.dtype not in _HALF or scales.dim() != 2:
        _refuse(scales, "scales", _HALF, dims=2)
    groups, K = scales.shape[1], 2 * half
    group = K // groups if groups else 128
    if group not in GROUPS or group * groups != K:      # (a multiple of group, then)
        raise ValueError(f"scales must have K / group columns, group one of {GROUPS}: K = {K}, scales "
                         f"{tuple(scales.shape)}")
    _full(scales, "scales", scales.dtype, (N, groups), codes.device)
    if zeros is None:
        return N, K, group, None
    _full(zeros, "zeros", scales.dtype, (N, groups), codes.device)
    return N, K, group, zeros.data_ptr()


def dequantize_w4(codes, scales, zeros: Optional[torch.Tensor] = None, out_dtype=torch.float32, out=None):
    """The weights that codes, scales and zeros stand for, N x K in `out_dtype`
    (fp32, fp16 or bf16)."""
    N, K, group, z = _w4(codes, scales, zeros)
    dev = codes.device
    out = _out(out, "out", (N, K), _out_dtype(out_dtype), dev)
    _call("lpgemm_dequantize_w4", dev, N, K, group, _HALF[scales.dtype], codes.data_ptr(), scales.data_ptr(), z,
          _TYPE[out_dtype], out.data_ptr())
    return out


def _x_and_w4(x, codes, scales, zeros):
    M, K, stride = _rows(x, "x", _HALF)
    N, Kw, group, z = _w4(codes, scales, zeros)
    if K != Kw:
        raise ValueError(f"K mismatch: x {tuple(x.shape)}, codes {tuple(codes.shape)}")
    if scales.dtype != x.dtype:
        raise TypeError(f"scales must have x's type {x.dtype}, got {scales.dtype}")
    if x.device != codes.device:
        raise ValueError("all tensors must be on the same device")
    return M, N, K, stride, group, z


def _scratch(bytes_needed: int, dev, workspace):
    """(address, bytes) of a workspace, and what keeps it alive until the call is made."""
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or workspace.dtype is not _U8 or workspace.dim() != 1 \
                or workspace.device != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous 1-D uint8 tensor on {dev}")
        if workspace.numel() < bytes_needed:
            raise ValueError(f"workspace must hold {bytes_needed} bytes, got {workspace.numel()}")
    elif bytes_needed > 0:
        workspace = _empty(bytes_needed, dtype=_U8, device=dev)
    else:
        return None, 0, None
    return workspace.data_ptr(), workspace.numel(), workspace


def w4_workspace_bytes(M: int, N: int, K: int, group_size: int, gated: bool = False) -> int:
    """Bytes of scratch that gemm_w4 (gated: gated_gemm_w4, N = 2F) needs on the
    current device (-1: sizes out of range)."""
    return _size("lpgemm_w4_workspace", M, N, K, group_size, int(gated))


def _w4_scratch(M, N, K, group, gated, dev, workspace):
    if M <= W4_SHORT_M:
        return None, 0, None
    return _scratch(_size_on(dev, "lpgemm_w4_workspace", M, N, K, group, gated), dev, workspace)


def gemm_w4(x, codes, scales, zeros: Optional[torch.Tensor] = None, out_dtype=None, out=None, workspace=None):
    """C = x . W^T for 4-bit weights W (N x K, as quantize_w4 makes them) and x,
    M x K fp16 or bf16 of the scales' type (contiguous rows, a row stride that is
    a multiple of 8); C is M x N in `out_dtype` (x's type, or fp32, fp16, bf16).
    Sums are in fp32; up to 384 rows the weights enter them exactly, beyond each
    is rounded once to x's type (for exact weights, pass x 384 rows at a time).
    `workspace`: uint8 scratch of
    w4_workspace_bytes(M, N, K, group) to use instead of a new allocation."""
    M, N, K, stride, group, z = _x_and_w4(x, codes, scales, zeros)
    dev, t = x.device, x.dtype
    out_dtype = t if out_dtype is None else _out_dtype(out_dtype)
    out = _out(out, "out", (M, N), out_dtype, dev)
    ws, ws_bytes, _alive = _w4_scratch(M, N, K, group, 0, dev, workspace)
    _call("lpgemm_w4", dev, M, N, K, group, _HALF[t], x.data_ptr(), stride, codes.data_ptr(), scales.data_ptr(), z,
          _TYPE[out_dtype], out.data_ptr(), ws, ws_bytes)
    return out


def gated_gemm_w4(x, codes, scales, zeros: Optional[torch.Tensor] = None, activation: str = "silu", out_dtype=None,
                  out=None, workspace=None):
    """act(x . G^T) * (x . U^T) for 4-bit weights whose first F of 2 F rows are G
    and the others U; act "silu" or "gelu" (its tanh form).  M x F, otherwise
    as gemm_w4."""
    M, N, K, stride, group, z = _x_and_w4(x, codes, scales, zeros)
    act = _activation(activation)
    if N % 2:
        raise ValueError(f"codes must hold the gate's and the up projection's rows, an even number, got {N}")
    dev, t, F = x.device, x.dtype, N // 2
    out_dtype = t if out_dtype is None else _out_dtype(out_dtype)
    out = _out(out, "out", (M, F), out_dtype, dev)
    ws, ws_bytes, _alive = _w4_scratch(M, N, K, group, 1, dev, workspace)
    _call("lpgemm_gated_w4", dev, M, F, K, group, _HALF[t], act, x.data_ptr(), stride, codes.data_ptr(),
          scales.data_ptr(), z, _TYPE[out_dtype], out.data_ptr(), ws, ws_bytes)
    return out


def gated_ffn_workspace_bytes(M: int, D: int, F: int) -> int:
    """Bytes of scratch that gated_ffn needs on the current device (-1: sizes out of range)."""
    return _size("lpgemm_gated_ffn_workspace", M, D, F)


def gated_ffn_backward_workspace_bytes(M: int, D: int, F: int) -> int:
    """Bytes of scratch that gated_ffn_backward needs on the current device (-1: sizes out of range)."""
    return _size("lpgemm_gated_ffn_backward_workspace", M, D, F)


def _block(x, w_gate_up, w_down):
    """Checks the block's operands: (M, D, F, x's row stride)."""
    M, D, stride = _rows(x, "x", _HALF)
    _operand(w_gate_up, "w_gate_up", x.dtype, 2)
    _operand(w_down, "w_down", x.dtype, 2)
    F = w_down.shape[1]
    if w_down.shape[0] != D or w_gate_up.shape != (2 * F, D):
        raise ValueError(f"w_gate_up must be 2F x D and w_down D x F: x {tuple(x.shape)}, w_gate_up "
                         f"{tuple(w_gate_up.shape)}, w_down {tuple(w_down.shape)}")
    if w_gate_up.device != x.device or w_down.device != x.device:
        raise ValueError("all tensors must be on the same device")
    return M, D, F, stride


def gated_ffn(x, w_gate_up, w_down, activation: str = "silu", keep: bool = False, out=None, gate_up_out=None,
              workspace=None):
    """The gated feed-forward block (act(x . G^T) * (x . U^T)) . w_down^T.

    x: M x D fp16 or bf16 (contiguous rows, a row stride that is a multiple of
    8); w_gate_up: 2F x D, G's rows before U's; w_down: D x F; all of one type,
    D and F multiples of 8.  act is "silu" or "gelu" (its tanh form).  Returns y,
    M x D; with `keep` (y, gate_up), gate_up = x . w_gate_up^T, M x 2F, which
    gated_ffn_backward takes: torch's automatic differentiation does not see this
    call, and y carries no gradient.  `workspace`: uint8 scratch of
    gated_ffn_workspace_bytes(M, D, F) to use instead of a new allocation."""
    M, D, F, stride = _block(x, w_gate_up, w_down)
    act = _activation(activation)
    dev, t = x.device, x.dtype
    if gate_up_out is not None and not keep:
        raise ValueError("gate_up_out goes with keep=True")
    out = _out(out, "out", (M, D), t, dev)
    gate_up = _out(gate_up_out, "gate_up_out", (M, 2 * F), t, dev) if keep else None
    ws, ws_bytes, _alive = _scratch(_size_on(dev, "lpgemm_gated_ffn_workspace", M, D, F), dev, workspace)
    _call("lpgemm_gated_ffn", dev, M, D, F, _HALF[t], act, x.data_ptr(), stride, w_gate_up.data_ptr(),
          w_down.data_ptr(), gate_up.data_ptr() if keep else None, out.data_ptr(), ws, ws_bytes)
    return (out, gate_up) if keep else out


def gated_ffn_backward(dy, x, w_gate_up, w_down, gate_up, activation: str = "silu", grad_dtype=None,
                       needs=(True, True, True), workspace=None):
    """Gradients of gated_ffn: (dx, dw_gate_up, dw_down) from dy (M x D, as x)
    and the gate_up that gated_ffn(..., keep=True) returned.  dx has x's type;
    the weights' gradients have `grad_dtype` (x's type, or torch.float32).
    `needs` says which of the three are wanted; the others are None.
    `workspace`: uint8 scratch of gated_ffn_backward_workspace_bytes(M, D, F) to
    use instead of a new allocation."""
    M, D, F, stride = _block(x, w_gate_up, w_down)
    act = _activation(activation)
    dev, t = x.device, x.dtype
    My, Dy, dy_stride = _rows(dy, "dy", (t,))
    if (My, Dy) != (M, D) or dy.device != dev:
        raise ValueError(f"dy must have x's shape {tuple(x.shape)} and be on {dev}")
    _full(gate_up, "gate_up", t, (M, 2 * F), dev)
    grad_dtype = t if grad_dtype is None else grad_dtype
    if grad_dtype is not t and grad_dtype is not _F32:
        raise TypeError(f"grad_dtype must be {t} or torch.float32, got {grad_dtype}")
    shapes = ((M, D), t), ((2 * F, D), grad_dtype), ((D, F), grad_dtype)
    if len(needs) != 3:
        raise ValueError("needs must say which of dx, dw_gate_up and dw_down are wanted")
    grads = [_empty(*s, dtype=d, device=dev) if n else None for n, (s, d) in zip(needs, shapes)]
    ws, ws_bytes, _alive = _scratch(_size_on(dev, "lpgemm_gated_ffn_backward_workspace", M, D, F), dev, workspace)
    _call("lpgemm_gated_ffn_backward", dev, M, D, F, _HALF[t], act, dy.data_ptr(), dy_stride, x.data_ptr(), stride,
          w_gate_up.data_ptr(), w_down.data_ptr(), gate_up.data_ptr(), _TYPE[grad_dtype],
          *[g.data_ptr() if g is not None else None for g in grads], ws, ws_bytes)
    return tuple(grads)
