"""Low-precision dense GEMM for AMD MI355X (gfx950).

C = A . B with INT8 and packed INT4 operands summed exactly in int32, FP16
operands summed in FP32, and an INT8 variant with per-row x per-column fp32
dequantisation; around them, the per-row int8 quantiser of fp16 activations
(W8A8), the INT4 path through the FP6 E3M2 matrix cores, split-K variants
for products with few output tiles, an fp64 GEMM emulated with exact INT8
GEMMs, the operators of a quantised expert layer (_moe.py), and 4-bit weights
with group scales and the gated feed-forward block (_ffn.py).  The work runs in
hand-written HIP kernels behind the C ABI of include/lpgemm.h; this package is
the torch-facing binding (see _binding.py), the in-tree build step (build.py)
and the seeded input generators (inputs.py).

The operators of a quantised expert layer (include/lpgemm_moe.h, bound in
_moe.py) stand beside the GEMMs: residual + RMSNorm and silu(gate) * up with
int8 rows, MXFP4 quantisation and product, and products grouped by expert.
So do 4-bit weights with group scales and the gated feed-forward block with
its gradients (include/lpgemm_ffn.h, bound in _ffn.py).
"""
from ._binding import (LpgemmError, auto_config, config_count, f64_emu_moduli, force_config, f64_emu_workspace_bytes, gemm_f16, gemm_f64_emu, gemm_f64_emu_noalloc, gemm_i4, gemm_i4_e3m2, gemm_i4_via_e3m2,  # noqa: F401
                       gemm_f16_splitk, gemm_i4_splitk, gemm_i8_dequant_splitk, gemm_i8_splitk,
                       gemm_i8, gemm_i8_dequant, gemm_i8_kxn, i4_to_e3m2, load_library, quantize_rows_f16,
                       splitk_workspace, splitk_workspace_bytes, status_string, version, w8a8_linear,
                       w8a8_linear_fused)

__all__ = ["LpgemmError", "gemm_i8", "gemm_i8_kxn", "gemm_i4", "gemm_f16", "gemm_i8_dequant",
           "quantize_rows_f16", "w8a8_linear", "w8a8_linear_fused", "i4_to_e3m2", "gemm_i4_e3m2", "gemm_i4_via_e3m2",
           "gemm_f64_emu", "gemm_f64_emu_noalloc", "f64_emu_moduli", "f64_emu_workspace_bytes",
           "gemm_i8_splitk", "gemm_i4_splitk", "gemm_f16_splitk", "gemm_i8_dequant_splitk",
           "splitk_workspace", "splitk_workspace_bytes",
           "load_library", "status_string", "version", "config_count", "force_config", "auto_config"]

# the expert-layer operators, imported with torch on their first use
_MOE = ("add_rmsnorm_quantize", "silu_mul_quantize", "quantize_mxfp4", "dequantize_mxfp4", "mxfp4_scale_stride",
        "gemm_mxfp4", "gemm_i8_dequant_grouped", "gemm_f16_grouped", "gemm_mxfp4_grouped", "grouped_config_count",
        "force_grouped_config", "grouped_auto_config")
# ... and those of 4-bit weights and of the gated feed-forward block
_FFN = ("quantize_w4", "dequantize_w4", "gemm_w4", "gated_gemm_w4", "gated_ffn", "gated_ffn_backward",
        "w4_workspace_bytes", "gated_ffn_workspace_bytes", "gated_ffn_backward_workspace_bytes", "ffn_config_count",
        "force_ffn_config")
__all__ += _MOE + _FFN


def __getattr__(name):
    if name in _MOE:
        from . import _moe as module
        names = _MOE
    elif name in _FFN:
        from . import _ffn as module
        names = _FFN
    else:
        raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
    for n in names:
        globals()[n] = getattr(module, n)
    return globals()[name]
