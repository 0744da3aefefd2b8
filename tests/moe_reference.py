"""Plain 64-bit references of the expert-layer operators, written from the
definitions in include/lpgemm_moe.h (numpy; torch only for bfloat16)."""
import numpy as np
import torch

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
TINY = 2.0 ** -100


def to64(t):
    """A torch tensor's values as float64 on the host."""
    return t.detach().cpu().to(torch.float64).numpy()


def rows_int8(z32):
    """Codes and a (the largest magnitude) of binary32 rows z, by the rule
    q = rne(z * (127 * (1 / a))), each operation in binary32; rows with a < 2^-100 or a non-finite
    value get codes 0."""
    assert z32.dtype == np.float32
    a = np.abs(z32).max(axis=1, initial=0.0).astype(np.float32)
    finite = np.isfinite(z32).all(axis=1)
    live = finite & (a >= np.float32(TINY))
    with np.errstate(all="ignore"):
        inv = np.where(live, np.float32(127) * (np.float32(1) / a), np.float32(0)).astype(np.float32)
        q = np.rint((z32 * inv[:, None]).astype(np.float32))
    q[~live] = 0
    return q.astype(np.int8), a, live, finite


def add_rmsnorm(x, r, w, eps):
    """(h in x's type, z in binary32, rstd in 64 bits)."""
    h = x if r is None else (x.float() + r.float()).to(x.dtype)
    h64 = to64(h)
    z = (h.float() * w.float()[None]).numpy()     # exact products of 16-bit values
    with np.errstate(all="ignore"):
        rstd = 1.0 / np.sqrt((h64 * h64).sum(axis=1) / max(h64.shape[1], 1) + eps)
    return h, z, rstd


def silu_mul(x):
    x = to64(x)
    k = x.shape[1] // 2
    g, u = x[:, :k], x[:, k:]
    with np.errstate(all="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def mx_quantize(x64):
    """(codes 0..15 per value, scale bytes per block) of rows x K values."""
    rows, K = x64.shape
    b = x64.reshape(rows, K // 32, 32)
    finite = np.isfinite(b).all(axis=2)
    a = np.where(finite, np.abs(b).max(axis=2, initial=0.0), 0.0)
    _, e = np.frexp(a)                            # a = m 2^e, m in [1/2, 1): floor(log2 a) = e - 1
    byte = np.where(a > 0, np.clip(e - 1 - 2 + 127, 0, 254), 0)
    v = np.where(finite[..., None], b, 0.0) / np.exp2(byte.astype(np.float64) - 127)[..., None]
    m = np.abs(v)
    code = np.zeros(m.shape, dtype=np.int64)
    for i in range(1, 8):                         # past the midpoint, or on it from an odd code
        mid = (E2M1[i - 1] + E2M1[i]) / 2
        code = np.where((m > mid) | ((m == mid) & (i % 2 == 0)), i, code)
    code = code + 8 * np.signbit(v)
    byte = np.where(finite, byte, 255)
    code[~finite] = 0
    return code.reshape(rows, K), byte


def mx_values(codes, scales, K):
    """Values of packed codes (.. x K/2 bytes) and scale bytes (the first K/32 count)."""
    c = np.empty((*codes.shape[:-1], K), dtype=np.int64)
    c[..., 0::2] = codes & 15
    c[..., 1::2] = codes >> 4
    v = E2M1[c & 7] * np.where(c >= 8, -1.0, 1.0)
    s = np.exp2(scales[..., :K // 32].astype(np.float64) - 127)
    s = np.where(scales[..., :K // 32] == 255, np.nan, s)
    return v * np.repeat(s, 32, axis=-1)


def mx_pack(code):
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def mx_random(rng, rows, K, spread=4):
    """Random packed codes and padded scale bytes (padding set to 255, which
    nothing may read)."""
    stride = (K // 32 + 15) // 16 * 16
    codes = rng.integers(0, 256, (rows, K // 2), dtype=np.uint8)
    scales = np.full((rows, stride), 255, dtype=np.uint8)
    scales[:, :K // 32] = rng.integers(127 - spread, 128 + spread, (rows, K // 32))
    return codes, scales


def random_offsets(rng, rows, groups, empty=()):
    """groups + 1 ascending offsets of a random split; groups in `empty` get no rows."""
    weight = rng.gamma(0.7, size=groups)
    weight[list(empty)] = 0
    counts = rng.multinomial(rows, weight / weight.sum())
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def group_of_rows(offsets, rows):
    g = np.full(rows, -1)
    for i in range(len(offsets) - 1):
        g[offsets[i]:offsets[i + 1]] = i
    return g
