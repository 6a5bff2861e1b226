"""Plain 64-bit forms of the dense layer's operators and the bounds that their
arithmetic allows (numpy, CPU).

Every output is checked through its rounding, which is monotonic: with the value
before it within e of the exact v, the result lies between the roundings of v - e
and v + e.
"""
import numpy as np
from scipy.special import ndtr

import expert_ref as ref

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
EPS24 = 2.0 ** -24


def up32(n):
    return -(-n // 32) * 32


def act(z, kind):
    """act(z), act'(z) and how far the kernels' fp32 forms may be from either.

    exp and 1 / x are good to 2^-22; the rounding of exp's argument a adds |a| 2^-22
    (two products and a rounded constant); GELU's polynomial is within 5.1e-7 < 2^-20.
    Where a slope subtracts (1 - g), that difference is good to 2^-22 absolutely.
    Values under the smallest normal number may be flushed to zero.
    """
    z = np.asarray(z, np.float64)
    tiny = 2.0 ** -120 * (1 + np.abs(z))
    if kind == "none":
        return z, np.ones_like(z), np.zeros_like(z), np.zeros_like(z)
    if kind == "relu":
        return np.maximum(z, 0), (z > 0) * 1.0, np.zeros_like(z), np.zeros_like(z)
    if kind == "gelu":
        below, dens = ndtr(z), np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
        r = 2.0 ** -19 + z * z * 2.0 ** -22
        return z * below, below + z * dens, np.abs(z) * below * r + tiny, (below + np.abs(z) * dens) * r + tiny
    u, du = (z, np.ones_like(z)) if kind == "silu" else (
        np.sqrt(8 / np.pi) * (z + 0.044715 * z ** 3), np.sqrt(8 / np.pi) * (1 + 3 * 0.044715 * z * z))
    with np.errstate(over="ignore"):
        g, g1 = 1 / (1 + np.exp(-u)), 1 / (1 + np.exp(u))
    r = 2.0 ** -19 + np.abs(u) * 2.0 ** -21
    h = z * g
    return h, g + h * g1 * du, np.abs(h) * r + tiny, (g + np.abs(h) * g1 * du) * r + np.abs(h) * du * 2.0 ** -22 * g + tiny


def to_bf16(v):
    """float64 -> the nearest bf16, ties to even, as float64."""
    v = np.asarray(v, np.float64)
    _, e = np.frexp(v)
    step = np.ldexp(1.0, np.maximum(e - 1, -126) - 7)
    out = np.round(v / step) * step
    return np.where(np.isfinite(v), out, v)


def check_bf16(got, v, e, what=""):
    bad = ~((to_bf16(v - e) <= got) & (got <= to_bf16(v + e)))
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}; first {np.argwhere(bad)[:3].tolist()}, " \
                          f"{got[bad][:3]} for {v[bad][:3]} within {np.broadcast_to(e, v.shape)[bad][:3]}"


def check_codes(codes, scales, v, e, fmt, what=""):
    """codes [R, ld] and scales [R, ld] of v [R, K] known to within e; whole blocks, the last one
    filled with zeros; what lies behind them (0xEE, 0xDD) left as it was."""
    R, K = v.shape
    whole = up32(K)
    pad = np.zeros((R, whole - K))
    v, e = np.hstack([v, pad]), np.hstack([np.broadcast_to(e, v.shape), pad])
    width = whole // 2 if fmt == "e2m1" else whole
    assert (codes[:, width:] == 0xEE).all() and (scales[:, whole // 32:] == 0xDD).all(), what
    codes, s = codes[:, :width], scales[:, :whole // 32].astype(int) - 127
    a = np.abs(v).reshape(R, -1, 32)
    d = e.reshape(R, -1, 32)
    ex = np.vectorize(lambda x: ref.scale_exponent(x, fmt), otypes=[int])
    lo, hi = (a - d).clip(0).max(-1), (a + d).max(-1)
    low = np.where(lo == 0, -127, ex(lo))
    ok = (low <= s) & (s <= ex(hi)) | (lo == 0) & (s == 0)
    assert ok.all(), f"{what}: scales {np.argwhere(~ok)[:3].tolist()}, {s[~ok][:3]} for {lo[~ok][:3]} to {hi[~ok][:3]}"
    got = ref.values(codes, (s + 127).astype(np.uint8), fmt)
    per = np.repeat(s, 32, axis=1)

    def rounded(x):
        c, neg = ref.to_codes(np.ldexp(x, -per), fmt)
        return np.ldexp(ref.GRIDS[fmt][c] * np.where(neg, -1, 1), per)

    ok = (rounded(v - e) <= got) & (got <= rounded(v + e))
    assert ok.all(), f"{what}: codes {np.argwhere(~ok)[:3].tolist()}, {got[~ok][:3]} for {v[~ok][:3]}"


def norm(x, w, b, eps):
    """y, mean, rstd of rows and the bounds of each, fp32 sums in chains of at most 48 roundings."""
    N = x.shape[1]
    mean = x.mean(1, keepdims=True)
    var = ((x - mean) ** 2).mean(1, keepdims=True)
    rstd = 1 / np.sqrt(var + eps)
    xhat = (x - mean) * rstd
    em = 48 * EPS24 * np.abs(x).mean(1, keepdims=True)
    er = 48 * EPS24 + em ** 2 / (var + eps)                # of rstd, relative
    ey = np.abs(w) * (em * rstd + np.abs(xhat) * (er + 4 * EPS24)) + 2 * EPS24 * (np.abs(xhat * w) + np.abs(b))
    return xhat * w + b, mean[:, 0], rstd[:, 0], ey, em[:, 0], (er * rstd)[:, 0]


def norm_backward(x, dy, mean, rstd, w, dres, blocks=304):
    """dx, dw, db from the given statistics, and their bounds."""
    T, N = x.shape
    mean, rstd = mean[:, None], rstd[:, None]
    xhat = (x - mean) * rstd
    g = dy * w
    s1, s2 = g.mean(1, keepdims=True), (g * xhat).mean(1, keepdims=True)
    dx = rstd * (g - s1 - xhat * s2) + dres
    chain = 48 * EPS24
    a1, a2 = np.abs(g).mean(1, keepdims=True), np.abs(g * xhat).mean(1, keepdims=True)
    ex = 2 * EPS24 * np.abs(xhat)
    edx = np.abs(rstd) * (chain * (a1 + np.abs(xhat) * a2) + np.abs(xhat) * 4 * EPS24 * a2 + 4 * EPS24 * (np.abs(g) + np.abs(s1) + np.abs(xhat * s2)))
    edx += ex * np.abs(rstd * s2) + 2 * EPS24 * (np.abs(dx) + np.abs(dres))
    chain = (T / blocks + 64) * EPS24
    return dx, (dy * xhat).sum(0), dy.sum(0), edx, chain * np.abs(dy * xhat).sum(0) + 2 * EPS24 * np.abs(dy * xhat).sum(0), \
        chain * np.abs(dy).sum(0)
