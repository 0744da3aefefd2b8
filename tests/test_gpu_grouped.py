"""GPU: products grouped by expert, and the MXFP4 product, against plain
64-bit references.

The int8 kind is exact: the int32 sum, two binary32 products, one rounding to
C's type.  The others are held to an error relative to sum |a||b|: one MFMA
adds 16 (binary16) or 64 (MXFP4) products to the accumulator, so a result
passes through K / 16 (K / 64) accumulations and a few more inside the
instruction and across waves, each within 2^-23; 16-bit C adds one rounding
of its own."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import moe_reference as ref  # noqa: E402
import precision_dense_gemm_02_amd as lp  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
OWN = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lp.load_library()


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def check_sums(got, exact, den, steps, t):
    """Results of type t against exact sums with sum |a||b| = den, where a
    result passed through `steps` accumulations.  binary16 has no room for
    sums past 65504, which become infinities of their sign: wherever the error
    bound allows either, both are right."""
    near = (steps + 8) * 2.0 ** -23 * den * (1 + OWN[t]) + OWN[t] * np.abs(exact) + 2.0 ** -24
    ok = np.abs(got - exact) <= near
    if t == "f16":
        ok |= np.isinf(got) & (np.sign(got) == np.sign(exact)) & (np.abs(exact) + near >= 65520)
    assert ok.all()


class Problem:
    """Operands of one grouped product and its reference."""

    def __init__(self, kind, tokens, groups, N, K, seed):
        self.kind, self.K, self.N = kind, K, N
        rng = self.rng = np.random.default_rng(seed)
        if kind == "i8":
            self.a = rng.integers(-128, 128, (tokens, K), dtype=np.int8)
            self.b = rng.integers(-128, 128, (groups, N, K), dtype=np.int8)
            self.rs = rng.uniform(1e-4, 1e-2, tokens).astype(np.float32)
            self.cs = rng.uniform(1e-4, 1e-2, (groups, N)).astype(np.float32)
            self.av, self.bv = self.a.astype(np.float64), self.b.astype(np.float64)
        elif kind == "f16":
            self.a = rng.standard_normal((tokens, K)).astype(np.float16)
            self.b = (rng.standard_normal((groups, N, K)) * 0.05).astype(np.float16)
            self.av, self.bv = self.a.astype(np.float64), self.b.astype(np.float64)
        else:
            self.a, self.as_ = ref.mx_random(rng, tokens, K)
            b, bs = ref.mx_random(rng, groups * N, K)
            self.b, self.bs = b.reshape(groups, N, b.shape[1]), bs.reshape(groups, N, bs.shape[1])
            self.av, self.bv = ref.mx_values(self.a, self.as_, K), ref.mx_values(self.b, self.bs, K)

    def run(self, offsets, index=None, t="f32", out=None):
        o, i = _dev(offsets), None if index is None else _dev(index)
        kw = dict(row_index=i, out_dtype=TYPES[t], out=out)
        if self.kind == "i8":
            return lp.gemm_i8_dequant_grouped(_dev(self.a), _dev(self.b), o, _dev(self.rs), _dev(self.cs), **kw)
        if self.kind == "f16":
            return lp.gemm_f16_grouped(_dev(self.a), _dev(self.b), o, **kw)
        return lp.gemm_mxfp4_grouped(_dev(self.a), _dev(self.as_), _dev(self.b), _dev(self.bs), o, **kw)

    def check(self, c, offsets, index=None, t="f32", rows=None):
        """C (on the GPU) against the reference, on the grouped rows."""
        got = ref.to64(c)
        n = got.shape[0]
        group = ref.group_of_rows(offsets, n)
        index = np.arange(n) if index is None else index
        for g in range(len(offsets) - 1):
            at = np.nonzero(group == g)[0]
            if not len(at):
                continue
            src = index[at]
            ok = (src >= 0) & (src < self.a.shape[0])
            a = np.where(ok[:, None], self.av[np.where(ok, src, 0)], 0.0)
            exact = a @ self.bv[g].T
            if self.kind == "i8":
                rs = np.where(ok, self.rs[np.where(ok, src, 0)], np.float32(0))
                want = (exact.astype(np.float32) * rs[:, None]) * self.cs[g][None]
                want = torch.from_numpy(want.astype(np.float32)).to(TYPES[t]).double().numpy()
                np.testing.assert_array_equal(got[at], want)
            else:
                den = np.abs(a) @ np.abs(self.bv[g]).T
                check_sums(got[at], exact, den, self.K / (16 if self.kind == "f16" else 64), t)


KINDS = ("i8", "f16", "mxfp4")
K_STEP = {"i8": 16, "f16": 8, "mxfp4": 32}

# rows, groups, N, K in steps of the kind's granularity: every kernel (8, 16
# and 32 row tiles; 64, 128 and 256 row tiles), K of one step, odd multiples
# and lengths past a few stages, N below, at and past a tile, N % 4 != 0
SHAPES = [(1, 1, 1, 1), (1, 4, 32, 5), (8, 64, 70, 33), (5, 3, 33, 64), (16, 2, 130, 40), (13, 5, 64, 31), (100, 7, 96, 65),
          (64, 2, 31, 128), (200, 4, 257, 20), (301, 6, 128, 37), (500, 4, 132, 16), (900, 5, 300, 50),
          (1500, 3, 510, 70), (2100, 4, 1028, 9), (700, 1, 4100, 24)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,groups,N,ksteps", SHAPES)
def test_grouped(kind, rows, groups, N, ksteps):
    K = ksteps * K_STEP[kind]
    t = ("f32", "f16", "bf16")[(rows + N) % 3]
    print("[case] grouped", kind, rows, groups, N, K, t, flush=True)
    tokens = max(1, rows // 3)
    p = Problem(kind, tokens, groups, N, K, seed=rows + N)
    offsets = ref.random_offsets(p.rng, rows, groups, empty=(1,) if groups > 2 else ())
    index = p.rng.integers(0, tokens, rows).astype(np.int32)
    p.check(p.run(offsets, index, t), offsets, index, t)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows", [7, 40, 260, 1200])
def test_rows_in_place_and_types(kind, rows):
    """No row_index: row i of C is row i of A; every type of C."""
    print("[case] plain rows", kind, rows, flush=True)
    K = 24 * K_STEP[kind]
    p = Problem(kind, rows, 3, 150, K, seed=rows)
    offsets = ref.random_offsets(p.rng, rows, 3)
    for t in TYPES:
        p.check(p.run(offsets, None, t), offsets, None, t)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,groups", [(6, 9), (50, 3), (300, 4), (700, 2)])
def test_rows_outside_groups_and_bad_routing(kind, rows, groups):
    """Rows before the first and past the last group stay as they were;
    indices outside A give zeros; offsets outside the rows are clamped;
    descending ones make empty groups."""
    print("[case] routing", kind, rows, groups, flush=True)
    K, N = 9 * K_STEP[kind], 66
    p = Problem(kind, 20, groups, N, K, seed=rows)
    index = p.rng.integers(0, 20, rows).astype(np.int32)
    index[[0, rows // 2, rows - 1]] = (-1, 20, 2 ** 31 - 1)
    inner = ref.random_offsets(p.rng, rows - 3, groups) + 2     # rows 0, 1 and the last belong to nobody
    out = torch.full((rows, N), -77.0, device="cuda")
    p.run(inner, index, out=out)
    p.check(out, inner, index)
    assert (out[:2] == -77).all() and (out[-1] == -77).all()
    wild = inner.copy()
    wild[0], wild[-1] = -5, rows + 1000
    p.check(p.run(wild, index), np.clip(wild, 0, rows), index)
    # one group of everything; then descending offsets: nothing is written
    one = np.array([0] * groups + [rows], dtype=np.int32)
    p.check(p.run(one, index), one, index)
    out.fill_(-77.0)
    p.run(np.arange(groups, -1, -1).astype(np.int32), index, out=out)
    assert (out == -77).all()


@pytest.mark.parametrize("kind", KINDS)
def test_many_groups(kind):
    """More groups than one scan of 64 covers, most of them empty."""
    for rows, groups in ((90, 300), (64, 64), (65, 65), (1000, 129)):
        print("[case] many groups", kind, rows, groups, flush=True)
        K = 5 * K_STEP[kind]
        p = Problem(kind, 30, groups, 40, K, seed=rows)
        offsets = ref.random_offsets(p.rng, rows, groups)
        index = p.rng.integers(0, 30, rows).astype(np.int32)
        p.check(p.run(offsets, index), offsets, index)


@pytest.mark.parametrize("kind", KINDS)
def test_empty_sizes(kind):
    p = Problem(kind, 4, 2, 40, K_STEP[kind], seed=1)
    zero = np.zeros(3, dtype=np.int32)
    assert p.run(zero, np.zeros(0, dtype=np.int32)).shape == (0, 40)
    z = Problem(kind, 4, 2, 40, 0, seed=1)                      # K = 0: an empty sum
    offsets = np.array([0, 3, 5], dtype=np.int32)
    index = np.array([0, 1, 2, 3, 0, 1], dtype=np.int32)
    out = torch.full((6, 40), 5.0, device="cuda")
    z.run(offsets, index, out=out)
    assert (out[:5] == 0).all() and (out[5] == 5).all()
    n = Problem(kind, 4, 2, 0, K_STEP[kind], seed=1)
    assert n.run(offsets, index).shape == (6, 0)
    e = Problem(kind, 0, 2, 40, K_STEP[kind], seed=1)           # no tokens: rows of zeros
    out.fill_(5.0)
    e.run(offsets, index, out=out)
    assert (out[:5] == 0).all() and (out[5] == 5).all()


def test_weights_and_results_past_4_gib():
    """Byte offsets past 2^32 in the weights and in C."""
    print("[case] 4.7 GB of weights", flush=True)
    G, N, K = 80, 14336, 4096
    g = torch.Generator(device="cuda").manual_seed(1)
    b = torch.randint(-128, 128, (G, N, K), dtype=torch.int8, device="cuda", generator=g)
    a = torch.randint(-128, 128, (40, K), dtype=torch.int8, device="cuda", generator=g)
    offsets = torch.zeros(G + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = 3
    offsets[G] = 40                                             # 3 rows in the first, 37 in the last group
    one = torch.ones(40, device="cuda")
    c = lp.gemm_i8_dequant_grouped(a, b, offsets, one, torch.ones(G, N, device="cuda"))
    for rows, w in ((slice(0, 3), b[0]), (slice(3, 40), b[G - 1])):
        assert torch.equal(c[rows], (a[rows].double() @ w.double().t()).float())
    del b, c
    print("[case] 5.2 GB of C", flush=True)
    rows, N, K = 80000, 16384, 64
    a = torch.randint(-128, 128, (rows, K), dtype=torch.int8, device="cuda", generator=g)
    b = torch.randint(-128, 128, (2, N, K), dtype=torch.int8, device="cuda", generator=g)
    offsets = torch.tensor([0, 100, rows], dtype=torch.int32, device="cuda")
    c = lp.gemm_i8_dequant_grouped(a, b, offsets, torch.ones(rows, device="cuda"), torch.ones(2, N, device="cuda"))
    for rows_, w in ((slice(0, 100), b[0]), (slice(rows - 100, rows), b[1])):
        assert torch.equal(c[rows_], (a[rows_].double() @ w.double().t()).float())


# every kernel at sizes that end inside its tile, its stage and its ring:
# rows of groups around every tile height and around the 32- and 64-row steps
# in which a partial tile of 128 and 256 rows runs; N below, at and past the
# tile widths and odd; K of one step to three more stages than the deepest
# ring holds, whole and partial
CONFIGS = range(11)
FORCED = [((1, 0, 7), 33, 1), ((8, 9, 16, 17), 70, 7), ((31, 33, 1, 64), 129, 31), ((65, 127, 128), 64, 17),
          ((129, 190, 3), 257, 40), ((255, 256, 60), 300, 9), ((257, 70, 320, 450), 260, 26), ((520, 5), 513, 12)]


@pytest.fixture(params=CONFIGS)
def forced(request):
    assert lp.grouped_config_count() == len(CONFIGS)
    previous = lp.force_grouped_config(request.param)
    yield request.param
    lp.force_grouped_config(previous)


@pytest.mark.parametrize("kind", KINDS)
def test_every_kernel(kind, forced):
    for counts, N, ksteps in FORCED:
        K = ksteps * K_STEP[kind]
        rows = sum(counts)
        t = ("f32", "f16", "bf16")[(rows + forced) % 3]
        print("[case] kernel", forced, kind, counts, N, K, t, flush=True)
        p = Problem(kind, 50, len(counts), N, K, seed=rows)
        offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        index = p.rng.integers(0, 50, rows).astype(np.int32)
        index[rows // 2] = 50                       # one row of zeros
        p.check(p.run(offsets, index, t), offsets, index, t)


@pytest.mark.parametrize("M", [1, 17, 64, 100, 190, 256, 330])
def test_every_kernel_mxfp4(M, forced):
    rng = np.random.default_rng(M)
    for N, K in ((31, 32), (260, 288), (513, 2080)):
        print("[case] mxfp4 kernel", forced, M, N, K, flush=True)
        a, as_ = ref.mx_random(rng, M, K)
        b, bs = ref.mx_random(rng, N, K)
        c = ref.to64(lp.gemm_mxfp4(_dev(a), _dev(as_), _dev(b), _dev(bs)))
        av, bv = ref.mx_values(a, as_, K), ref.mx_values(b, bs, K)
        check_sums(c, av @ bv.T, np.abs(av) @ np.abs(bv).T, K / 64, "f32")


def test_every_kernel_mxfp4_scales(forced):
    """Scales of every size, NaN scales and padding bytes in every kernel."""
    test_mxfp4_scales_of_every_size(300)
    test_mxfp4_nan_scale(200)


@pytest.mark.parametrize("kind", KINDS)
def test_every_kernel_k_zero_and_untouched_rows(kind, forced):
    test_empty_sizes(kind)
    test_rows_outside_groups_and_bad_routing(kind, 300, 4)


@pytest.mark.parametrize("kind", KINDS)
def test_every_kernel_rows_without_a_token(kind, forced):
    """A row_index outside A gives zeros also where the weights or their
    scales are infinite or NaN; so does a product without tokens."""
    for counts, N, ksteps in (((3, 1), 33, 3), ((40, 70, 5), 96, 9), ((300,), 130, 8)):
        K, rows = ksteps * K_STEP[kind], sum(counts)
        print("[case] no token", forced, kind, counts, N, K, flush=True)
        p = Problem(kind, 50, len(counts), N, K, seed=rows)
        bad = np.arange(1, N, 3)
        if kind == "i8":
            p.cs[:, bad] = np.array([np.inf, np.nan, -np.inf], dtype=np.float32)[bad % 3]
        elif kind == "f16":
            p.b[:, bad, K // 2] = np.array([np.inf, np.nan, -np.inf], dtype=np.float16)[bad % 3]
        else:
            p.bs[:, bad, 0] = 255
        offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        index = p.rng.integers(0, 50, rows).astype(np.int32)
        absent = np.unique(np.concatenate([[0, rows - 1], p.rng.integers(0, rows, rows // 3)]))
        index[absent] = p.rng.choice([-1, 50, -2 ** 31, 2 ** 31 - 1], len(absent))
        with_token = np.setdiff1d(np.arange(rows), absent)
        for t in TYPES:
            c = p.run(offsets, index, t).cpu()
            assert (c[absent] == 0).all()
            assert (~c[with_token][:, bad].isfinite()).all()
            assert c[with_token][:, np.setdiff1d(np.arange(N), bad)].isfinite().all()
        p.a = p.a[:0]
        if kind == "i8":
            p.rs = p.rs[:0]
        elif kind == "mxfp4":
            p.as_ = p.as_[:0]
        assert (p.run(offsets, index) == 0).all()


# ------------------------------------------------------------ MXFP4 product

MX_SHAPES = [(1, 1, 32), (1, 33, 64), (16, 70, 4096), (9, 300, 544), (33, 100, 96), (64, 129, 2880), (100, 257, 1024),
             (130, 64, 320), (200, 260, 32 * 45), (513, 300, 256), (700, 4100, 96), (2300, 1030, 288)]


@pytest.mark.parametrize("M,N,K", MX_SHAPES)
def test_mxfp4(M, N, K):
    t = ("f32", "f16", "bf16")[(M + N) % 3]
    print("[case] mxfp4", M, N, K, t, flush=True)
    rng = np.random.default_rng(M + N + K)
    a, as_ = ref.mx_random(rng, M, K)
    b, bs = ref.mx_random(rng, N, K)
    c = ref.to64(lp.gemm_mxfp4(_dev(a), _dev(as_), _dev(b), _dev(bs), out_dtype=TYPES[t]))
    av, bv = ref.mx_values(a, as_, K), ref.mx_values(b, bs, K)
    exact, den = av @ bv.T, np.abs(av) @ np.abs(bv).T
    check_sums(c, exact, den, K / 64, t)


@pytest.mark.parametrize("M", [5, 40, 300, 1100])
def test_mxfp4_scales_of_every_size(M):
    """Scales across the whole byte range whose product stays in binary32:
    each block's own scale counts, in the row and the block it belongs to."""
    rng = np.random.default_rng(M)
    N, K = 300 if M < 1000 else 1100, 1088
    a, as_ = ref.mx_random(rng, M, K)
    b, bs = ref.mx_random(rng, N, K)
    as_[:, :K // 32] = rng.integers(20, 230, (M, K // 32))
    bs[:, :K // 32] = (250 - as_[0, :K // 32])[None]
    as_[:, :K // 32] = np.clip(as_[0, :K // 32][None].astype(int) + rng.integers(-8, 9, (M, K // 32)), 0, 254)
    c = ref.to64(lp.gemm_mxfp4(_dev(a), _dev(as_), _dev(b), _dev(bs)))
    av, bv = ref.mx_values(a, as_, K), ref.mx_values(b, bs, K)
    exact, den = av @ bv.T, np.abs(av) @ np.abs(bv).T
    assert (np.abs(c - exact) <= (K / 64 + 8) * 2.0 ** -23 * den).all()


@pytest.mark.parametrize("M", [3, 50, 200, 1100])
def test_mxfp4_nan_scale(M):
    """A scale byte of 255 makes its row of A (column of B) NaN, no other."""
    rng = np.random.default_rng(M)
    N, K = 600 if M > 1000 else 70, 416
    a, as_ = ref.mx_random(rng, M, K)
    b, bs = ref.mx_random(rng, N, K)
    as_[M // 2, 3] = 255
    bs[N - 1, K // 32 - 1] = 255
    c = lp.gemm_mxfp4(_dev(a), _dev(as_), _dev(b), _dev(bs)).cpu()
    nan = torch.zeros(M, N, dtype=torch.bool)
    nan[M // 2] = True
    nan[:, N - 1] = True
    assert torch.equal(c.isnan(), nan)


def test_mxfp4_empty():
    a, s = torch.zeros(3, 0, dtype=torch.uint8, device="cuda"), torch.zeros(3, 0, dtype=torch.uint8, device="cuda")
    assert (lp.gemm_mxfp4(a, s, a, s) == 0).all()
    a, s = torch.zeros(0, 16, dtype=torch.uint8, device="cuda"), torch.zeros(0, 16, dtype=torch.uint8, device="cuda")
    assert lp.gemm_mxfp4(a, s, a, s).shape == (0, 0)


@pytest.mark.parametrize("M,N,K", [(1, 40, 64), (17, 70, 96), (130, 300, 2080), (300, 513, 8192)])
def test_every_kernel_mxfp4_bit_for_bit(M, N, K, forced):
    """With one scale for all blocks the products are multiples of a quarter,
    up to 36, and every partial sum fits 24 bits (36 x 8192 x 4 < 2^24): C is
    the exact sum, rounded once to its type."""
    rng = np.random.default_rng(M + K)
    a, as_ = ref.mx_random(rng, M, K, spread=0)
    b, bs = ref.mx_random(rng, N, K, spread=0)
    exact = torch.from_numpy(ref.mx_values(a, as_, K) @ ref.mx_values(b, bs, K).T)
    offsets = np.array([0, M], dtype=np.int32)
    for t in TYPES:
        print("[case] bit for bit", forced, M, N, K, t, flush=True)
        want = exact.to(TYPES[t])
        assert torch.equal(lp.gemm_mxfp4(_dev(a), _dev(as_), _dev(b), _dev(bs), out_dtype=TYPES[t]).cpu(), want)
        assert torch.equal(lp.gemm_mxfp4_grouped(_dev(a), _dev(as_), _dev(b[None]), _dev(bs[None]), _dev(offsets),
                                                 out_dtype=TYPES[t]).cpu(), want)


@pytest.mark.parametrize("sa,sb", [(0, 254), (254, 0), (0, 130), (130, 0), (1, 253), (254, 20)])
def test_every_kernel_mxfp4_first_and_last_scale(sa, sb, forced):
    """Scale bytes at both ends, 2^-127 and 2^127, with codes of every value,
    where the products stay in binary32: exact."""
    for M, N, K in ((3, 70, 96), (200, 130, 288)):
        print("[case] scale ends", forced, sa, sb, M, N, K, flush=True)
        rng = np.random.default_rng(M)
        a, as_ = ref.mx_random(rng, M, K, spread=0)
        b, bs = ref.mx_random(rng, N, K, spread=0)
        as_[:, :K // 32], bs[:, :K // 32] = sa, sb
        c = ref.to64(lp.gemm_mxfp4(_dev(a), _dev(as_), _dev(b), _dev(bs)))
        np.testing.assert_array_equal(c, ref.mx_values(a, as_, K) @ ref.mx_values(b, bs, K).T)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,groups", [(700, 5000), (3000, 65536)])
def test_thousands_of_groups(kind, rows, groups):
    """Up to the most groups there may be: 1024 scans of 64."""
    print("[case] thousands of groups", kind, rows, groups, flush=True)
    K = K_STEP[kind]
    p = Problem(kind, 30, groups, 9, K, seed=rows)
    offsets = ref.random_offsets(p.rng, rows, groups)
    index = p.rng.integers(0, 30, rows).astype(np.int32)
    p.check(p.run(offsets, index), offsets, index)
    last = np.zeros(groups + 1, dtype=np.int32)      # all of them in the last group
    last[-1] = rows
    p.check(p.run(last, index), last, index)


# ------------------------------------------------- streams, graphs, repeats

def test_other_stream_and_graph_replay():
    """The operators on a stream of their own, then captured into a graph and
    replayed with eager work in between: bit for bit the same."""
    rng = np.random.default_rng(3)
    p = Problem("i8", 40, 6, 200, 256, seed=3)
    offsets = ref.random_offsets(rng, 120, 6)
    index = rng.integers(0, 40, 120).astype(np.int32)
    x = torch.randn(40, 256, device="cuda").half()
    w = torch.randn(256, device="cuda").half()
    b, o, i, cs = _dev(p.b), _dev(offsets), _dev(index), _dev(p.cs)
    wq = lp.quantize_mxfp4(torch.randn(100, 224, device="cuda").half())
    torch.cuda.synchronize()

    def layer():
        q, s, h = lp.add_rmsnorm_quantize(x, w, 1e-6, residual=x)
        y = lp.gemm_i8_dequant_grouped(q, b, o, s, cs, row_index=i, out_dtype=torch.float16)
        q2, s2 = lp.silu_mul_quantize(y[:, :192])
        m = lp.quantize_mxfp4(h[:, :224])
        return q, s, h, y, q2, s2, *m, lp.gemm_mxfp4(*m, *wq)

    want = [v.clone() for v in layer()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = layer()
    side.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = layer()
    for _ in range(3):
        for v in captured:
            v.zero_()
        graph.replay()
        eager = layer()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(captured, want))
        assert all(torch.equal(u, v) for u, v in zip(eager, want))
