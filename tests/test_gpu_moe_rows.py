"""GPU: residual + RMSNorm and silu(gate) * up with int8 rows, and MXFP4
quantisation, against plain 64-bit references.

The norm's codes, h and the MXFP4 codes are defined value by value (no sum
enters them), so they must match exactly.  Derived tolerances:
  norm scale   the sum of squares adds at most K / 64 + 16 roundings in a row
               (per lane, then across lanes and waves), each 2^-24 relative,
               halved by the square root; four more operations follow
  activation   exp(-g) through exp2: the argument's rounding costs |g| 2^-24
               relative, the exponential, the reciprocal and three products
               about 8 roundings: z is within (1.5 |g| + 16) 2^-24 of exact
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import moe_reference as ref  # noqa: E402
import precision_dense_gemm_02_amd as lp  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
ULP = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lp.load_library()


def _case(*a):
    print("[case]", *a, flush=True)


def _rows(M, K, dtype, seed, big_columns=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g) * torch.exp2(torch.rand(M, 1, generator=g) * 8 - 4)
    if big_columns and K:
        x[:, torch.randint(0, K, (max(1, K // 100),), generator=g)] *= 10
    return x.to(dtype)


def _check_norm(x, r, w, eps, q, s, h):
    """x, r, w on the host; q, s, h from the GPU."""
    eh, z, rstd = ref.add_rmsnorm(x, r, w, eps)
    assert torch.equal(h.cpu().view(torch.int16), eh.view(torch.int16))
    eq, a, live, finite = ref.rows_int8(z)
    np.testing.assert_array_equal(q.cpu().numpy(), eq)
    s = s.cpu().numpy().astype(np.float64)
    want = np.where(live, a.astype(np.float64) / 127 * rstd, 0.0)
    tol = (x.shape[1] / 64 + 16 + 8) * ULP
    assert (np.abs(s - want)[finite] <= tol * want[finite]).all()
    assert np.isnan(s[~finite]).all()


# one token to more rows than SIMDs; K through every register variant (one
# chunk of 8 to 16384), the two-pass kernel beyond, and odd multiples of 8
NORM_SHAPES = [(1, 8), (1, 4096), (3, 264), (7, 1000), (2, 2056), (5, 8192), (2, 8200), (3, 16384), (2, 16392),
               (2, 40000), (1025, 512), (1030, 520), (1024, 1032), (1027, 2048), (1100, 4104), (1024, 8192)]


@pytest.mark.parametrize("t", sorted(TYPES))
@pytest.mark.parametrize("M,K", NORM_SHAPES)
def test_norm(M, K, t):
    _case("norm", M, K, t)
    x, r = _rows(M, K, TYPES[t], 1), _rows(M, K, TYPES[t], 2)
    w = _rows(1, K, TYPES[t], 3, False)[0]
    q, s, h = lp.add_rmsnorm_quantize(x.cuda(), w.cuda(), 1e-6, residual=r.cuda())
    _check_norm(x, r, w, 1e-6, q, s, h)
    q, s, h = lp.add_rmsnorm_quantize(x.cuda(), w.cuda(), 1e-5)
    _check_norm(x, None, w, 1e-5, q, s, h)


@pytest.mark.parametrize("t", sorted(TYPES))
@pytest.mark.parametrize("M,K", [(3, 512), (1100, 256), (2, 16400)])
def test_norm_special_rows(M, K, t):
    """Zero rows, infinities, NaN, and rows whose squares overflow."""
    _case("norm special", M, K, t)
    x = _rows(max(M, 6), K, TYPES[t], 4)
    x[0] = 0
    x[1, 5] = float("inf")
    x[2, K - 1] = float("nan")
    w = _rows(1, K, TYPES[t], 3, False)[0]
    if t == "bf16":
        x[3] = 1e30       # the sum of squares leaves binary32
        x[4] = 1e-38      # the products with the weights fall below 2^-100
    q, s, h = lp.add_rmsnorm_quantize(x.cuda(), w.cuda(), 1e-6)
    s, q = s.cpu(), q.cpu()
    assert s[0] == 0 and (q[0] == 0).all()
    assert s[1:3].isnan().all() and (q[1:3] == 0).all()
    if t == "bf16":
        assert s[3].isnan() and (q[3] == 0).all() and s[4] == 0 and (q[4] == 0).all()
    rest = slice(5, None)
    _check_norm(x[rest], None, w, 1e-6, q[rest], s[rest], h[rest])


@pytest.mark.parametrize("M,K", [(5, 768), (1030, 264), (2, 16400)])
def test_norm_strides_and_in_place(M, K):
    _case("norm strides", M, K)
    x, r = _rows(M, K, torch.float16, 5), _rows(M, K, torch.float16, 6)
    w = _rows(1, K, torch.float16, 3, False)[0]
    big = torch.full((3, M, K + 24), 7.0, dtype=torch.float16, device="cuda")
    big[0, :, 8:8 + K] = x.cuda()
    big[1, :, 16:16 + K] = r.cuda()
    keep = big.clone()
    q, s, h = lp.add_rmsnorm_quantize(big[0, :, 8:8 + K], w.cuda(), 1e-6, residual=big[1, :, 16:16 + K],
                                      residual_out=big[2, :, :K])
    _check_norm(x, r, w, 1e-6, q, s, h)
    keep[2, :, :K] = h
    assert torch.equal(big, keep)        # nothing outside h was written
    for into in (0, 1):                  # h over x, h over the residual
        bx, br = x.cuda(), r.cuda()
        q, s, h = lp.add_rmsnorm_quantize(bx, w.cuda(), 1e-6, residual=br, residual_out=(bx, br)[into])
        assert h is (bx, br)[into]
        _check_norm(x, r, w, 1e-6, q, s, h)


@pytest.mark.parametrize("eps", [0.0, 1e-44, 2.0 ** -110, 1e-25])
@pytest.mark.parametrize("K", [64, 512, 1024, 2048, 4096, 8192, 16384, 32768, 32776])
def test_norm_rows_whose_squares_underflow(K, eps):
    """Rows from 2^-98 up to 2^-40, whose squares are subnormal or zero in
    binary32, with an eps that does not hide them."""
    _case("norm underflow", K, eps)
    g = torch.Generator().manual_seed(K)
    size = torch.exp2(torch.tensor([-98., -90, -80, -74, -70, -66, -63, -60, -55, -52, -50, -49, -45, -40]))
    x = (torch.randn(len(size), K, generator=g) * size[:, None]).to(torch.bfloat16)
    r = (torch.randn(len(size), K, generator=g) * size[:, None]).to(torch.bfloat16)
    w = _rows(1, K, torch.bfloat16, 3, False)[0]
    eps = float(np.float32(eps))
    q, s, h = lp.add_rmsnorm_quantize(x.cuda(), w.cuda(), eps, residual=r.cuda())
    _check_norm(x, r, w, eps, q, s, h)
    # large weights on the smallest values
    w = torch.full((K,), 2.0 ** 60, dtype=torch.bfloat16)
    x = torch.exp2(torch.randint(-133, -120, (3, K), generator=g).float()).to(torch.bfloat16)
    q, s, h = lp.add_rmsnorm_quantize(x.cuda(), w.cuda(), eps)
    _check_norm(x, None, w, eps, q, s, h)


def test_norm_rows_past_4_gib():
    """Row offsets past 2^32 bytes, in a stream whose rows lie far apart."""
    M, K, stride = 2200, 512, 1 << 20
    _case("norm far rows", M, K, stride)
    big = torch.empty((M, stride), dtype=torch.bfloat16, device="cuda")
    x, r = _rows(M, K, torch.bfloat16, 7), _rows(M, K, torch.bfloat16, 8)
    w = _rows(1, K, torch.bfloat16, 3, False)[0]
    big[:, :K] = x.cuda()
    q, s, h = lp.add_rmsnorm_quantize(big[:, :K], w.cuda(), 1e-6, residual=r.cuda(), residual_out=big[:, K:2 * K])
    _check_norm(x, r, w, 1e-6, q, s, h)


def test_more_rows_than_one_launch():
    """Past 2^21 rows, in two launches: the rows around the seam and the last."""
    M, K = (1 << 21) + 5, 16
    _case("many rows", M, K)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(M, K, generator=g, device="cuda").half()
    r = torch.randn(M, K, generator=g, device="cuda").half()
    w = _rows(1, K, torch.float16, 3, False)[0]
    q, s, h = lp.add_rmsnorm_quantize(x, w.cuda(), 1e-6, residual=r)
    for part in (slice(0, 9), slice((1 << 21) - 4, M)):
        _check_norm(x[part].cpu(), r[part].cpu(), w, 1e-6, q[part], s[part], h[part])
    q, s = lp.silu_mul_quantize(x)
    for part in (slice(0, 9), slice((1 << 21) - 4, M)):
        _check_silu(x[part].cpu(), q[part], s[part])


def test_norm_no_rows_no_columns():
    w = torch.ones(64, dtype=torch.float16, device="cuda")
    q, s, h = lp.add_rmsnorm_quantize(torch.empty(0, 64, dtype=torch.float16, device="cuda"), w, 1e-6)
    assert q.shape == (0, 64) and s.shape == (0,) and h.shape == (0, 64)
    q, s, _ = lp.add_rmsnorm_quantize(torch.empty(5, 0, dtype=torch.float16, device="cuda"), w[:0], 1e-6)
    assert (s.cpu() == 0).all()
    q, s = lp.silu_mul_quantize(torch.empty(5, 0, dtype=torch.float16, device="cuda"))
    assert q.shape == (5, 0) and (s.cpu() == 0).all()


def _check_silu(x, q, s):
    z = ref.silu_mul(x)
    g = np.abs(ref.to64(x)[:, :z.shape[1]])
    finite = np.isfinite(z).all(axis=1)
    q, s = q.cpu().numpy().astype(np.float64), s.cpu().numpy().astype(np.float64)
    assert np.isnan(s[~finite]).all() and (q[~finite] == 0).all()
    z, g, q, s = z[finite], g[finite], q[finite], s[finite]
    a = np.abs(z).max(axis=1, initial=0.0)
    tol = (1.5 * g + 16) * ULP
    at = tol.max(axis=1, initial=0.0)      # also bounds the error of the largest value
    assert (np.abs(s - a / 127) <= (at + 2 * ULP) * a / 127).all()
    zero = a < ref.TINY
    assert (s[zero] == 0).all() and (q[zero] == 0).all()
    with np.errstate(all="ignore"):
        exact = np.where(zero[:, None], 0.0, z / (a / 127)[:, None])
    assert (np.abs(q - exact) <= 0.5 + np.abs(exact) * (tol + at[:, None] + 4 * ULP)).all()


@pytest.mark.parametrize("t", sorted(TYPES))
@pytest.mark.parametrize("M,K", NORM_SHAPES)
def test_silu_mul(M, K, t):
    _case("silu", M, K, t)
    x = _rows(M, 2 * K, TYPES[t], 9)
    q, s = lp.silu_mul_quantize(x.cuda())
    _check_silu(x, q, s)


@pytest.mark.parametrize("t", sorted(TYPES))
def test_silu_mul_special_rows(t):
    x = _rows(6, 2 * 512, TYPES[t], 10)
    x[0] = 0
    x[1, 3] = float("nan")
    x[2, 600] = float("inf")
    x[3, :512] = -1000        # exp(-g) overflows: silu is -0
    x[4, :512:2] = 60         # saturated gates
    q, s = lp.silu_mul_quantize(x.cuda())
    _check_silu(x, q, s)
    assert s.cpu()[0] == 0 and s.cpu()[3] == 0


@pytest.mark.parametrize("t", sorted(TYPES))
def test_silu_mul_every_gate(t):
    """Every finite 16-bit gate, alone in its row, against 64 bits.  In units
    of 2^-24: the exponential 2, its remainder's factor 1, the sum with one 1,
    the reciprocal 2, two products and the scale's division 1 each: 8, here 9;
    below -86 the reciprocal is subnormal, 2^-149 in 2^-128, 4 more.  Where
    exp(-g) leaves binary32 (g < -88.723) the quotient is -0; a largest value
    below 2^-100 counts as zero, one above binary32 gives NaN."""
    g = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(TYPES[t])
    g = g[g.isfinite()]
    for up in (1.0, 3.0e4, 1e30) if t == "bf16" else (1.0, 65504.0):
        _case("every gate", t, up)
        x = torch.zeros(len(g), 16, dtype=TYPES[t])
        x[:, 0], x[:, 8] = g, up
        q, s = lp.silu_mul_quantize(x.cuda())
        q, s = q.cpu(), s.cpu().double()
        g64 = g.double()
        z = torch.where(g64 < -88.723, 0.0, g64 / (1 + torch.exp(-g64))) * x[:, 8].double()
        a = z.abs()
        zero, past, live = a < ref.TINY * 0.999, a > 3.4029e38, (a > ref.TINY * 1.001) & (a < 3.4027e38)
        assert (s[zero] == 0).all() and (q[zero] == 0).all()
        assert s[past].isnan().all() and (q[past] == 0).all()
        bound = torch.where(g64 < -86, 13.0, 9.0) * ULP
        assert ((s * 127 - a).abs() <= bound * a)[live].all()
        assert torch.equal(q[live][:, 0], (127 * torch.sign(z[live])).to(torch.int8))


def test_silu_mul_strided():
    x = _rows(33, 2 * 136, torch.bfloat16, 11)
    big = torch.full((33, 2 * 136 + 40), float("nan"), dtype=torch.bfloat16, device="cuda")
    big[:, 8:8 + 272] = x.cuda()
    q, s = lp.silu_mul_quantize(big[:, 8:8 + 272])
    _check_silu(x, q, s)


# on both sides of every change of the number of wavefronts per row and of
# chunks per lane, and of the register form; more rows than CUs, too
FORMS = [512, 520, 1024, 1032, 2048, 2056, 4096, 4104, 8192, 8200, 16384, 16392, 32768, 32776]


@pytest.mark.parametrize("t", sorted(TYPES))
@pytest.mark.parametrize("K", FORMS)
def test_row_forms(K, t):
    for M in (1, 3, 300):
        _case("row forms", M, K, t)
        x, r = _rows(M, K, TYPES[t], 12), _rows(M, K, TYPES[t], 13)
        w = _rows(1, K, TYPES[t], 3, False)[0]
        q, s, h = lp.add_rmsnorm_quantize(x.cuda(), w.cuda(), 1e-6, residual=r.cuda())
        _check_norm(x, r, w, 1e-6, q, s, h)
        bx = x.cuda()                                   # h over x
        q, s, h = lp.add_rmsnorm_quantize(bx, w.cuda(), 1e-6, residual=r.cuda(), residual_out=bx)
        _check_norm(x, r, w, 1e-6, q, s, h)
        if M > 3:
            continue
        x = _rows(M, 2 * K, TYPES[t], 14)
        q, s = lp.silu_mul_quantize(x.cuda())
        _check_silu(x, q, s)


@pytest.mark.parametrize("K", FORMS)
def test_row_forms_special_rows(K):
    """The row's largest value, an infinity or a NaN in any wavefront's part."""
    _case("row forms special", K)
    at = sorted({0, 7, 511 % K, 512 % K, K // 2, K - 9, K - 1})
    x = torch.zeros(3 * len(at) + 1, K, dtype=torch.bfloat16)
    for i, k in enumerate(at):
        x[3 * i, k], x[3 * i + 1, k], x[3 * i + 2, k] = 2.0, float("inf"), float("nan")
    w = torch.ones(K, dtype=torch.bfloat16)
    for up in (None, torch.ones(K, dtype=torch.bfloat16)):
        if up is None:
            q, s, _ = lp.add_rmsnorm_quantize(x.cuda(), w.cuda(), 0.0)
        else:
            q, s = lp.silu_mul_quantize(torch.cat([x, up.expand_as(x)], 1).cuda())
        q, s = q.cpu(), s.cpu()
        for i, k in enumerate(at):
            want = torch.zeros(K, dtype=torch.int8)
            want[k] = 127
            assert torch.equal(q[3 * i], want) and s[3 * i] > 0
            assert s[3 * i + 1].isnan() and s[3 * i + 2].isnan() and (q[3 * i + 1:3 * i + 3] == 0).all()
        assert s[-1] == 0 and (q[-1] == 0).all()


# ------------------------------------------------------------------ MXFP4

def _check_mx(x, codes, scales):
    code, byte = ref.mx_quantize(ref.to64(x))
    blocks = byte.shape[1]
    got = scales.cpu().numpy()
    np.testing.assert_array_equal(got[:, :blocks], byte)
    assert (got[:, blocks:] == 0).all()
    np.testing.assert_array_equal(codes.cpu().numpy(), ref.mx_pack(code))


@pytest.mark.parametrize("t", sorted(TYPES))
@pytest.mark.parametrize("M,K", [(1, 32), (1, 4096), (3, 96), (5, 544), (33, 2880), (257, 1024), (7, 32 * 333)])
def test_quantize_mxfp4(M, K, t):
    _case("mx", M, K, t)
    x = _rows(M, K, TYPES[t], 12)
    codes, scales = lp.quantize_mxfp4(x.cuda())
    _check_mx(x, codes, scales)
    for out in (torch.float32, torch.float16, torch.bfloat16):
        y = lp.dequantize_mxfp4(codes, scales, out_dtype=out)
        want = torch.from_numpy(ref.mx_values(codes.cpu().numpy(), scales.cpu().numpy(), K)).to(out)
        assert torch.equal(y.cpu(), want)


@pytest.mark.parametrize("t", sorted(TYPES))
def test_quantize_mxfp4_every_value(t):
    """Every finite 16-bit value, in a block whose largest value is itself,
    twice and eight times it (where finite): ties, subnormals, both ends."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    v = bits.view(TYPES[t])
    v = v[v.isfinite()]
    x = torch.zeros(v.numel(), 96, dtype=TYPES[t])
    for b, factor in enumerate((1, 2, 8)):
        top = v.double().abs() * factor
        ok = top <= torch.finfo(TYPES[t]).max
        x[:, 32 * b + 7] = v
        x[:, 32 * b + 30] = torch.where(ok, top, v.double()).to(TYPES[t])
        x[:, 32 * b + 11] = -v / 3
    codes, scales = lp.quantize_mxfp4(x.cuda())
    _check_mx(x, codes, scales)


@pytest.mark.parametrize("t", sorted(TYPES))
def test_mxfp4_special_blocks(t):
    x = _rows(4, 256, TYPES[t], 13)
    x[0, :32] = 0
    x[1, 40] = float("inf")
    x[2, 100] = float("nan")
    x[3, 64:96] = -0.0
    codes, scales = lp.quantize_mxfp4(x.cuda())
    _check_mx(x, codes, scales)
    y = lp.dequantize_mxfp4(codes, scales).cpu()
    assert y[1, 32:64].isnan().all() and y[2, 96:128].isnan().all()
    assert not y[0].isnan().any() and not y[3].isnan().any() and (y[0, :32] == 0).all()


def test_dequantize_mxfp4_every_code_and_scale():
    codes = np.tile(np.arange(256, dtype=np.uint8), (256, 1))          # K = 512
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 16, axis=1)
    y = lp.dequantize_mxfp4(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()).cpu()
    want = torch.from_numpy(ref.mx_values(codes, scales, 512)).float()
    assert torch.equal(y[:255], want[:255]) and y[255].isnan().all()


def test_quantize_mxfp4_strided():
    x = _rows(50, 224, torch.float16, 14)
    big = torch.full((50, 280), float("nan"), dtype=torch.float16, device="cuda")
    big[:, 24:248] = x.cuda()
    codes, scales = lp.quantize_mxfp4(big[:, 24:248])
    _check_mx(x, codes, scales)


@pytest.mark.parametrize("t", sorted(TYPES))
@pytest.mark.parametrize("M,K", [(4096, 8192), (4105, 8224)])
def test_mxfp4_many_values(M, K, t):
    """From 2^25 values on a lane handles two chunks: the same codes, scales
    and values as a few rows at a time, and the rows at both ends checked."""
    _case("mx many", M, K, t)
    x = torch.randn(M, K, device="cuda").to(TYPES[t])
    codes, scales = lp.quantize_mxfp4(x)
    for rows in (slice(0, 3), slice(M - 3, M)):
        _check_mx(x[rows].cpu(), codes[rows], scales[rows])
    y = {d: lp.dequantize_mxfp4(codes, scales, out_dtype=d) for d in (torch.float32, torch.float16, torch.bfloat16)}
    for r in range(0, M, 1500):
        part = slice(r, min(r + 1500, M))
        c, s = lp.quantize_mxfp4(x[part])
        assert torch.equal(codes[part], c) and torch.equal(scales[part], s)
        for d in y:
            assert torch.equal(y[d][part], lp.dequantize_mxfp4(c, s, out_dtype=d))
