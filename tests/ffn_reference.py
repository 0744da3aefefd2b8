"""Plain 64-bit references of the operators in include/lpgemm_ffn.h, written
from its definitions, and how far a kernel's results may be from them.

Bounds: a binary32 sum of n terms in any order is within n U of the sum of the
magnitudes (U = 2^-23: half a step is 2^-24, and a matrix instruction may cut
instead of rounding); a rounding to type t is within eps(t) / 2 of the value, or
half the smallest step where it is subnormal."""
import math

import torch

U = 2.0 ** -23
C0, C1 = math.sqrt(2 / math.pi), 0.044715


def half_step(v, dtype):
    """The most that rounding v to dtype changes it."""
    if dtype is torch.float32:
        return v.abs() * 2.0 ** -24 + 2.0 ** -150
    return v.abs() * (torch.finfo(dtype).eps / 2) + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def rounded(v, err, dtype):
    """The error of a value known to `err` once it is rounded to dtype."""
    return err + half_step(v.abs() + err, dtype)


def act(g, kind):
    a = g if kind == "silu" else 2 * C0 * (g + C1 * g ** 3)
    return g * torch.sigmoid(a)


def act_slope(g, kind):
    if kind == "silu":
        p, q = torch.sigmoid(g), torch.sigmoid(-g)
        return p + g * p * q
    a = 2 * C0 * (g + C1 * g ** 3)
    p, q = torch.sigmoid(a), torch.sigmoid(-a)
    return p + g * p * q * 2 * C0 * (1 + 3 * C1 * g ** 2)


# |act'| is at most 1.13, |act''| at most 1; the kernels' activation is within
# 24 units of 2^-24 of the formula (12 of the logistic function, the argument's
# and two products'), its derivative within 32 of 2^-24 (1 + |g|)
MOST_SLOPE, MOST_BEND = 1.13, 1.0
ACT_ERR, SLOPE_ERR = 24 * 2.0 ** -24, 32 * 2.0 ** -24


def unpack(codes):
    """int64 codes -8..7, N x K, of packed bytes (the even k in the low nibble)."""
    n = torch.stack([codes.long() % 16, codes.long() // 16], -1).reshape(codes.shape[0], -1)
    return torch.where(n >= 8, n - 16, n)


def pack(code):
    n = code.long() % 16
    return (n[:, 0::2] + 16 * n[:, 1::2]).to(torch.uint8)


def spread(t, group):
    return t.double().repeat_interleave(group, dim=1)


def w4_values(codes, scales, zeros, group):
    z = 0.0 if zeros is None else spread(zeros, group)
    return (unpack(codes).double() - z) * spread(scales, group)


W4_EXACT_ROWS = 384          # beyond, the weights are rounded to x's type first


def w4_product(x, codes, scales, zeros, group, rounded_weights=None):
    """(x . W^T, the error of the kernel's binary32 sums).  With weights rounded
    to x's type each is off by at most half a step, |x| . half_step(W) in all, and
    the sums are of K products of them."""
    t = x.dtype
    x = x.double()
    M, K = x.shape
    if rounded_weights or (rounded_weights is None and M > W4_EXACT_ROWS):
        w = w4_values(codes, scales, zeros, group)
        # (code - zero and its product with the scale are rounded to binary32 before that: 2^-23 of the weight)
        off = half_step(w, t) + 2.0 ** -23 * w.abs()
        return x @ w.t(), x.abs() @ off.t() + (K + 40) * U * (x.abs() @ (w.abs() + off).t())
    z = torch.zeros_like(scales).double() if zeros is None else zeros.double()
    s = spread(scales, group).abs()
    # x (24 + code) is summed over a group, then (24 + zero) sum x taken off
    parts = x.abs() @ ((24 + unpack(codes).double()) * s + (24 + spread(z, group)).abs() * s).t()
    depth = group + 4 + K // group + 16
    return x @ w4_values(codes, scales, zeros, group).t(), depth * U * parts


def gated(y, err, kind):
    """(act(gate) * up, its error) from both projections' sums and theirs."""
    F = y.shape[1] // 2
    g, u, dg, du = y[:, :F], y[:, F:], err[:, :F], err[:, F:]
    a = act(g, kind)
    da = MOST_SLOPE * dg + ACT_ERR * (a.abs() + dg)
    h = a * u
    return h, da * (u.abs() + du) + a.abs() * du + 2.0 ** -23 * h.abs()


def product(a, b, da=None, db=None):
    """(a . b, error of a binary32 sum of operands known to da and db)."""
    K = a.shape[1]
    size = a.abs() @ b.abs()
    err = (K + 40) * U * size          # (40: the splits and the waves' sums)
    if da is not None:
        err = err + da @ b.abs()
    if db is not None:
        err = err + (a.abs() + (0 if da is None else da)) @ db
    return a @ b, err


def block(x, w_gate_up, w_down, kind):
    """((y, error), (gate_up, error)) before their rounding."""
    t = x.dtype
    gu, dgu = product(x.double(), w_gate_up.double().t())
    h, dh = gated(gu, dgu, kind)
    return product(h, w_down.double().t(), rounded(h, dh, t)), (gu, dgu)


def block_backward(dy, x, w_gate_up, w_down, gate_up, kind):
    """((dx, error), (dw_gate_up, error), (dw_down, error)) before their rounding."""
    t = x.dtype
    F = w_down.shape[1]
    dh, e = product(dy.double(), w_down.double())
    g, u = gate_up[:, :F].double(), gate_up[:, F:].double()
    a, slope = act(g, kind), act_slope(g, kind)
    da, ds = ACT_ERR * a.abs(), SLOPE_ERR * (1 + g.abs())
    dg, du, h = dh * u * slope, dh * a, a * u
    dg_err = rounded(dg, e * u.abs() * (slope.abs() + ds) + dh.abs() * u.abs() * ds + 2.0 ** -23 * dg.abs(), t)
    du_err = rounded(du, e * (a.abs() + da) + dh.abs() * da + 2.0 ** -24 * du.abs(), t)
    h_err = rounded(h, da * u.abs() + 2.0 ** -24 * h.abs(), t)
    dgu, dgu_err = torch.cat([dg, du], 1), torch.cat([dg_err, du_err], 1)
    return (product(dgu, w_gate_up.double(), dgu_err),
            product(dgu.t(), x.double(), dgu_err.t()),
            product(dy.double().t(), h, None, h_err))


def check(got, want, err, what=""):
    """got, rounded once from a value within err of want."""
    assert got.shape == want.shape, (what, got.shape, want.shape)
    off = (got.double() - want).abs()
    limit = rounded(want, err, got.dtype)
    bad = ~(off <= limit)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst " \
                          f"{float((off / limit).nan_to_num(1e30).max()):.3g} times the bound at " \
                          f"{[int(v) for v in bad.nonzero()[0]]}"
