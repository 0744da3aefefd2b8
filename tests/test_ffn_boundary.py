"""The entry points of 4-bit weights and of the gated feed-forward block
without a GPU: exported, and refusing bad arguments on the host before any HIP
call (fake pointers are never dereferenced by validation); then the Python
binding's own refusals, and the workspaces' sizes."""
import re

import pytest

torch = pytest.importorskip("torch")

import precision_dense_gemm_02_amd as lp  # noqa: E402
from precision_dense_gemm_02_amd import _binding as b  # noqa: E402
from precision_dense_gemm_02_amd import _ffn, _moe  # noqa: E402

P = 0x10000           # 256-byte aligned, never dereferenced
INVALID, MISALIGNED, SHAPE = b.LPGEMM_ERROR_INVALID_VALUE, b.LPGEMM_ERROR_MISALIGNED, b.LPGEMM_ERROR_UNSUPPORTED_SHAPE
HEADER = b.HEADER_PATH.replace("lpgemm.h", "lpgemm_ffn.h")
F16, BF16 = torch.float16, torch.bfloat16

DEFAULTS = {
    "lpgemm_quantize_w4": dict(N=4, K=128, group=64, type=1, W=P, w_stride=128, codes=P, scales=P, zeros=P),
    "lpgemm_dequantize_w4": dict(N=4, K=128, group=64, type=1, codes=P, scales=P, zeros=P, out_type=0, Y=P),
    "lpgemm_w4": dict(M=8, N=4, K=128, group=64, type=2, X=P, x_stride=128, codes=P, scales=P, zeros=P, out_type=0,
                      C=P, workspace=P, workspace_bytes=1 << 30),
    "lpgemm_gated_w4": dict(M=8, F=4, K=128, group=64, type=2, activation=1, X=P, x_stride=128, codes=P, scales=P,
                            zeros=P, out_type=0, H=P, workspace=P, workspace_bytes=1 << 30),
    "lpgemm_gated_ffn": dict(M=8, D=128, F=64, type=1, activation=0, X=P, x_stride=128, W_gate_up=P, W_down=P, GU=P,
                             Y=P, workspace=P, workspace_bytes=1 << 30),
    "lpgemm_gated_ffn_backward": dict(M=8, D=128, F=64, type=1, activation=0, dY=P, dy_stride=128, X=P, x_stride=128,
                                      W_gate_up=P, W_down=P, GU=P, grad_type=0, dX=P, dW_gate_up=P, dW_down=P,
                                      workspace=P, workspace_bytes=1 << 30),
}
W4 = [n for n in sorted(DEFAULTS) if n.endswith("_w4")]
W4_PRODUCTS = ["lpgemm_w4", "lpgemm_gated_w4"]
BLOCK = ["lpgemm_gated_ffn", "lpgemm_gated_ffn_backward"]
SIZES = {"M", "N", "K", "F", "D"}
STRIDES = {"w_stride", "x_stride", "dy_stride"}


def call(name, **kw):
    args = dict(DEFAULTS[name])
    assert set(kw) <= set(args), kw
    args.update(kw)
    return _moe._function(name)(*args.values(), None)


def header():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_exports_every_declared_symbol():
    text = header()
    names = re.findall(r"^lpgemm_status\s+(lpgemm_\w+)\s*\(", text, flags=re.M)
    assert set(names) == set(DEFAULTS) == set(_ffn._SIGNATURES)
    assert set(_ffn._SIGNATURES) <= set(_moe._SIGNATURES_ELSEWHERE)
    for n in names:
        args = re.search(n + r"\s*\((.*?)\)\s*;", text, flags=re.S).group(1)
        declared = [re.search(r"(\w+)$", a.strip()).group(1) for a in args.split(",")]
        assert declared == [*DEFAULTS[n], "stream"], n
        # (a pointer, an int64_t or an enum, in the places the binding has them)
        kinds = [_moe._p if "*" in a or "hipStream_t" in a else _moe._i64 if "int64_t" in a else _moe._int
                 for a in args.split(",")]
        assert kinds == _ffn._SIGNATURES[n], n
    for n in re.findall(r"(lpgemm_\w+)\s*\(", text):
        assert hasattr(b.load_library(), n), n


def test_constants_agree():
    constants = dict(re.findall(r"#define (LPGEMM_\w+) (\d+)", header()))
    assert int(constants["LPGEMM_W4_SHORT_M"]) == _ffn.W4_SHORT_M
    assert constants["LPGEMM_W4_EXACT_M"] in lp.gemm_w4.__doc__
    for name in ("quantize_w4", "dequantize_w4", "gemm_w4", "gated_gemm_w4", "gated_ffn", "gated_ffn_backward",
                 "w4_workspace_bytes", "gated_ffn_workspace_bytes", "gated_ffn_backward_workspace_bytes"):
        assert name in lp.__all__ and getattr(lp, name).__doc__


@pytest.mark.parametrize("name", sorted(DEFAULTS))
def test_sizes(name):
    args = DEFAULTS[name]
    for size in set(args) & (SIZES | {"group", "workspace_bytes"}):
        assert call(name, **{size: -8}) == INVALID, size
    for size in set(args) & {"M", "N"}:
        assert call(name, **{size: 2 ** 31}) == INVALID, size
    for t in (-1, 0, 3):        # 16-bit tensors only
        assert call(name, type=t) == INVALID
    for t in (-1, 3):
        if "out_type" in args:
            assert call(name, out_type=t) == INVALID
    for a in (-1, 2):
        if "activation" in args:
            assert call(name, activation=a) == INVALID
    if "grad_type" in args:
        for own, other in ((1, 2), (2, 1), (1, 3), (1, -1)):
            assert call(name, type=own, grad_type=other) == INVALID


@pytest.mark.parametrize("name", W4)
def test_groups(name):
    for group in (0, 1, 16, 48, 96, 512):
        assert call(name, group=group) == SHAPE, group
    for K, group in ((32, 64), (96, 64), (160, 128), (128, 256), (1048576 + 64, 64)):
        strides = {s: 2 * K for s in STRIDES & set(DEFAULTS[name])}
        assert call(name, K=K, group=group, **strides) == SHAPE, (K, group)


@pytest.mark.parametrize("name", BLOCK)
def test_block_sizes(name):
    strides = {s: 2 ** 19 for s in STRIDES & set(DEFAULTS[name])}
    for size in ("D", "F"):
        for bad in (4, 12, 132, 262144 + 8):
            assert call(name, **{size: bad}, **strides) == SHAPE, (size, bad)
    assert call(name, M=2 ** 31 - 256) == SHAPE
    assert call(name, M=2 ** 30) == SHAPE                      # 2^24 tiles of 64 x 64 of M x 2 F
    assert call(name, M=2 ** 24, D=4096, **{**strides}) == SHAPE
    assert call(name, D=262144, F=262144, **strides) == SHAPE


@pytest.mark.parametrize("name", W4_PRODUCTS)
def test_largest_products(name):
    n = "N" if name == "lpgemm_w4" else "F"
    assert call(name, M=134217728 + 1) == SHAPE
    assert call(name, **{n: 16777216 + 8}) == SHAPE
    assert call(name, M=2 ** 21, **{n: 2 ** 15}) == SHAPE


@pytest.mark.parametrize("name,stride", [(n, s) for n in sorted(DEFAULTS) for s in sorted(STRIDES & set(DEFAULTS[n]))])
def test_strides(name, stride):
    least = DEFAULTS[name][stride]
    for bad in (least - 8, 0, -least, least + 4):
        assert call(name, **{stride: bad}) == SHAPE, bad
    if name != "lpgemm_quantize_w4":
        assert call(name, **{stride: 2097152 + 8}) == SHAPE


@pytest.mark.parametrize("name", sorted(DEFAULTS))
def test_null_and_misaligned_pointers(name):
    optional = {"zeros", "GU", "dX", "dW_gate_up", "dW_down", "workspace"} if name != "lpgemm_gated_ffn_backward" \
        else {"dX", "dW_gate_up", "dW_down"}
    for k, v in DEFAULTS[name].items():
        if v != P:
            continue
        if k not in optional:
            assert call(name, **{k: None}) == INVALID, k
        by = 1 if k in ("scales", "zeros") else 128 if k == "workspace" else 8
        assert call(name, **{k: P + by}) == MISALIGNED, k
    if name == "lpgemm_gated_ffn":
        assert call(name, workspace=None) == INVALID


@pytest.mark.parametrize("name", sorted(DEFAULTS))
def test_empty_problems_read_nothing(name):
    args = DEFAULTS[name]
    nothing = {k: None for k, v in args.items() if v == P}
    empty = {"lpgemm_quantize_w4": ["N", "K"], "lpgemm_dequantize_w4": ["N", "K"], "lpgemm_w4": ["M", "N"],
             "lpgemm_gated_w4": ["M", "F"], "lpgemm_gated_ffn": ["M"], "lpgemm_gated_ffn_backward": ["D"]}[name]
    for size in empty:
        assert call(name, **{size: 0}, **nothing) == 0, size
        # the shape rules still hold
        if "group" in args:
            assert call(name, **{size: 0}, **nothing, group=48) == SHAPE
        else:
            assert call(name, **{size: 0}, **nothing, F=12) == SHAPE
    if name == "lpgemm_gated_ffn_backward":
        assert call(name, dX=None, dW_gate_up=None, dW_down=None) == 0      # nothing wanted
        assert call(name, M=0, F=0, **nothing) == 0


def test_workspace_sizes_out_of_range():
    lib = b.load_library()
    assert lp.w4_workspace_bytes(0, 64, 128, 64) == 0 and lp.w4_workspace_bytes(64, 0, 128, 64) == 0
    for bad in ((-1, 4, 128, 64, 0), (4, -1, 128, 64, 0), (4, 4, -64, 64, 0), (4, 4, 128, 48, 0), (4, 4, 96, 64, 0),
                (134217729, 4, 128, 64, 0), (4, 16777217, 128, 64, 0), (4, 5, 128, 64, 1)):
        assert lp.w4_workspace_bytes(*bad) == -1, bad
    for f in (lp.gated_ffn_workspace_bytes, lp.gated_ffn_backward_workspace_bytes):
        for bad in ((-1, 64, 64), (4, -8, 64), (4, 64, -8), (4, 12, 64), (4, 64, 12), (2 ** 31, 64, 64),
                    (2 ** 30, 64, 64), (4, 262152, 64)):
            assert f(*bad) == -1, bad
    assert lib.lpgemm_ffn_config_count() == lp.ffn_config_count() == 7


TOO_MANY_TILES = [(2 ** 21, 2 ** 15), (2 ** 15, 2 ** 21), (134217728, 512), (4096, 16777216)]   # 2^24 of 64 x 64


def test_products_of_too_many_tiles():
    for M, N in TOO_MANY_TILES:
        assert call("lpgemm_w4", M=M, N=N) == SHAPE
        assert call("lpgemm_gated_w4", M=M, F=N // 2) == SHAPE


def test_pinned_kernels():
    n = lp.ffn_config_count()
    assert lp.force_ffn_config(n) == -1 and lp.force_ffn_config(2) == -1
    assert lp.force_ffn_config(-1) == 2 and lp.force_ffn_config(-1) == -1


class _OnGpu(torch.Tensor):
    """A host tensor that says it is on a GPU, for the checks in front of a call."""
    is_cuda = property(lambda self: True)


def gpu(*shape, dtype=F16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(_OnGpu)


def w4(N=6, K=128, group=64, dtype=F16):
    return gpu(N, K // 2, dtype=torch.uint8), gpu(N, K // group, dtype=dtype)


def refused(kind, match, f, *args, **kw):
    with pytest.raises(kind, match=match):
        f(*args, **kw)


def test_binding_refuses_host_tensors():
    x, w = torch.zeros(4, 128, dtype=F16), torch.zeros(6, 64, dtype=torch.uint8)
    refused(ValueError, "GPU", lp.quantize_w4, x)
    refused(ValueError, "GPU", lp.dequantize_w4, w, torch.zeros(6, 2, dtype=F16))
    refused(ValueError, "GPU", lp.gemm_w4, x, *w4())
    refused(ValueError, "GPU", lp.gated_ffn, x, gpu(16, 128), gpu(128, 8))
    refused(TypeError, "torch.Tensor", lp.gated_ffn_backward, [1], gpu(4, 128), gpu(16, 128), gpu(128, 8), gpu(4, 16))


def test_binding_refuses_types():
    x = gpu(4, 128)
    codes, scales = w4()
    refused(TypeError, "w must be", lp.quantize_w4, x.float())
    refused(TypeError, "codes must be", lp.gemm_w4, x, codes.to(torch.int8), scales)
    refused(TypeError, "scales must be", lp.gemm_w4, x, codes, scales.float())
    refused(TypeError, "scales must have x's type", lp.gemm_w4, x, codes, scales.to(BF16).as_subclass(_OnGpu))
    refused(TypeError, "zeros must be", lp.gemm_w4, x, codes, scales, scales.float())
    refused(TypeError, "out_dtype", lp.gemm_w4, x, codes, scales, out_dtype=torch.int32)
    refused(TypeError, "w_gate_up must be", lp.gated_ffn, x, gpu(16, 128, dtype=BF16), gpu(128, 8))
    refused(TypeError, "w_down must be", lp.gated_ffn, x, gpu(16, 128), gpu(128, 8, dtype=torch.float32))
    block = gpu(4, 128), gpu(4, 128), gpu(16, 128), gpu(128, 8), gpu(4, 16)
    refused(TypeError, "grad_dtype", lp.gated_ffn_backward, *block, grad_dtype=BF16)
    refused(TypeError, "gate_up must be", lp.gated_ffn_backward, *block[:4], gpu(4, 16, dtype=BF16))


def test_binding_refuses_shapes():
    x = gpu(4, 128)
    codes, scales = w4()
    for group in (0, 16, 48, 512, 256):
        refused(ValueError, "group_size", lp.quantize_w4, x, group)
    refused(ValueError, "zeros=True", lp.quantize_w4, x, 64, zeros_out=gpu(4, 2))
    refused(ValueError, "codes_out", lp.quantize_w4, x, 64, codes_out=gpu(4, 32, dtype=torch.uint8))
    refused(ValueError, "scales must have", lp.dequantize_w4, codes, gpu(6, 3))
    refused(ValueError, "scales must have", lp.dequantize_w4, codes, gpu(6, 0))
    refused(ValueError, "scales must have shape", lp.dequantize_w4, codes, gpu(5, 2))
    refused(ValueError, "zeros must have shape", lp.gemm_w4, x, codes, scales, gpu(6, 1))
    refused(ValueError, "K mismatch", lp.gemm_w4, gpu(4, 64), codes, scales)
    refused(ValueError, "out must have shape", lp.gemm_w4, x, codes, scales, out=gpu(4, 5))
    refused(ValueError, "an even number", lp.gated_gemm_w4, x, *w4(5))
    refused(ValueError, "activation", lp.gated_gemm_w4, x, codes, scales, activation="relu")
    refused(ValueError, "workspace", _ffn._scratch, 512, torch.device("cpu"), torch.zeros(256, dtype=torch.uint8))
    refused(ValueError, "workspace", _ffn._scratch, 512, torch.device("cpu"), torch.zeros(512, dtype=torch.int8))
    refused(ValueError, "2F x D", lp.gated_ffn, x, gpu(16, 64), gpu(128, 8))
    refused(ValueError, "2F x D", lp.gated_ffn, x, gpu(24, 128), gpu(128, 8))
    refused(ValueError, "2F x D", lp.gated_ffn, x, gpu(16, 128), gpu(64, 8))
    refused(ValueError, "activation", lp.gated_ffn, x, gpu(16, 128), gpu(128, 8), activation="Silu")
    refused(ValueError, "keep=True", lp.gated_ffn, x, gpu(16, 128), gpu(128, 8), gate_up_out=gpu(4, 16))
    block = gpu(4, 128), x, gpu(16, 128), gpu(128, 8), gpu(4, 16)
    refused(ValueError, "dy must have", lp.gated_ffn_backward, gpu(5, 128), *block[1:])
    refused(ValueError, "gate_up must have", lp.gated_ffn_backward, *block[:4], gpu(4, 8))
    refused(ValueError, "needs", lp.gated_ffn_backward, *block, needs=(True, True))


def test_binding_refuses_more_scales_than_values():
    """... of which a group would hold none."""
    for half in (0, 1):
        codes, scales = gpu(6, half, dtype=torch.uint8), gpu(6, 3)
        refused(ValueError, "scales must have", lp.dequantize_w4, codes, scales)
        refused(ValueError, "scales must have", lp.gemm_w4, gpu(4, 2 * half), codes, scales)
        refused(ValueError, "scales must have", lp.gated_gemm_w4, gpu(4, 2 * half), codes, scales, gpu(6, 3))


def test_binding_refuses_columns_that_are_not_adjacent():
    for bad in (torch.zeros(4, 256, dtype=F16)[:, ::2], torch.zeros(128, 4, dtype=F16).t(),
                torch.zeros(4, 1, dtype=F16).expand(4, 128)):
        bad = bad.as_subclass(_OnGpu)
        for name, f in (("w", lambda: lp.quantize_w4(bad)), ("x", lambda: lp.gemm_w4(bad, *w4())),
                        ("x", lambda: lp.gated_gemm_w4(bad, *w4())),
                        ("x", lambda: lp.gated_ffn(bad, gpu(16, 128), gpu(128, 8))),
                        ("dy", lambda: lp.gated_ffn_backward(bad, gpu(4, 128), gpu(16, 128), gpu(128, 8), gpu(4, 16)))):
            refused(ValueError, f"the rows of {name} must be contiguous", f)
    # weights and codes are whole arrays
    refused(ValueError, "codes must be contiguous", lp.dequantize_w4, gpu(6, 128, dtype=torch.uint8)[:, :64], gpu(6, 2))
    refused(ValueError, "scales must be contiguous", lp.dequantize_w4, w4()[0], gpu(6, 4)[:, :2])
    refused(ValueError, "w_gate_up must be contiguous", lp.gated_ffn, gpu(4, 128), gpu(128, 16).t(), gpu(128, 8))
    refused(ValueError, "w_down must be contiguous", lp.gated_ffn, gpu(4, 128), gpu(16, 128), gpu(8, 128).t())


@pytest.mark.gpu
@pytest.mark.parametrize("M", [40, 600])
def test_workspace_that_is_too_small(M):
    """One byte less than asked for is refused, in both layers; nothing is written."""
    D, F = 1024, 512
    x, wgu, wd = (torch.randn(*s, device="cuda").half() for s in ((M, D), (2 * F, D), (D, F)))
    need = lp.gated_ffn_workspace_bytes(M, D, F)
    back = lp.gated_ffn_backward_workspace_bytes(M, D, F)
    codes, scales = lp.quantize_w4(wgu)
    w4_need = lp.w4_workspace_bytes(M, 2 * F, D, 128)
    assert need > 0 and back > 0 and (w4_need > 0 or M < 384)
    ws = torch.zeros(max(need, back, w4_need), dtype=torch.uint8, device="cuda")
    y, gu = lp.gated_ffn(x, wgu, wd, keep=True)
    out = torch.full_like(y, 7.0)
    p = lambda t: t.data_ptr()
    refused(ValueError, "workspace must hold", lp.gated_ffn, x, wgu, wd, workspace=ws[:need - 1])
    refused(ValueError, "workspace must hold", lp.gated_ffn_backward, y, x, wgu, wd, gu, workspace=ws[:back - 1])
    assert _moe._function("lpgemm_gated_ffn")(M, D, F, 1, 0, p(x), D, p(wgu), p(wd), None, p(out), p(ws), need - 1, None) == INVALID
    assert _moe._function("lpgemm_gated_ffn_backward")(M, D, F, 1, 0, p(y), D, p(x), D, p(wgu), p(wd), p(gu), 1, p(out),
                                                       None, None, p(ws), back - 1, None) == INVALID
    if w4_need:
        refused(ValueError, "workspace must hold", lp.gemm_w4, x, codes, scales, workspace=ws[:w4_need - 1])
        assert _moe._function("lpgemm_w4")(M, 2 * F, D, 128, 1, p(x), D, p(codes), p(scales), None, 1, p(out), p(ws),
                                           w4_need - 1, None) == INVALID
        assert _moe._function("lpgemm_w4")(M, 2 * F, D, 128, 1, p(x), D, p(codes), p(scales), None, 1, p(out), None,
                                           0, None) == INVALID
    torch.cuda.synchronize()
    assert (out == 7).all() and (ws == 0).all()


@pytest.mark.gpu
def test_no_workspace_for_products_that_are_refused():
    """(On a GPU: without one the size is -1 in any case.)"""
    for M, N in TOO_MANY_TILES:
        for gated in (False, True):
            assert lp.w4_workspace_bytes(M, N, 256, 64, gated) == -1, (M, N)
            assert lp.w4_workspace_bytes(M - 64, N, 256, 64, gated) > 0, (M, N)
