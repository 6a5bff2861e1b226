"""The dense layer as a whole and its gradients in 64 bits, each value with a bound
of how far the kernels' may be from it (numpy, CPU).

A value is (v, e): the kernels' lies within e of v.  A rounding is monotonic, so
rounded values lie between the roundings of v - e and v + e (``rounded_bf16``,
``Rounded``); a product adds 2^-20 of its sum of magnitudes.  ``Loose`` takes each
quantisation as an error of its own instead and leaves v as it is: with it the
formulas are those of the layer in real numbers.
"""
import numpy as np

import dense_ref as dr
import expert_ref as ref
from dense_ref import EPS24

ACC = 2.0 ** -20


def rounded_bf16(v, e):
    lo, hi = dr.to_bf16(v - e), dr.to_bf16(v + e)
    return (lo + hi) / 2, (hi - lo) / 2


def _exponents(a, fmt):
    ex = np.vectorize(lambda x: ref.scale_exponent(x, fmt), otypes=[int])
    return np.where(a == 0, -127, ex(a))


class Rounded:
    """Values as the kernels round them."""
    bf16 = staticmethod(rounded_bf16)

    @staticmethod
    def codes(v, e, fmt):
        """Blocks of 32 along the rows, the last one of each row cut."""
        R, K = v.shape
        pad = np.zeros((R, dr.up32(K) - K))
        w, d = np.hstack([v, pad]), np.hstack([np.broadcast_to(e, v.shape), pad])
        a, b = np.abs(w).reshape(R, -1, 32), d.reshape(R, -1, 32)
        ends = []
        for edge in ((a - b).clip(0).max(-1), (a + b).max(-1)):
            s = np.repeat(_exponents(edge, fmt), 32, axis=1)
            for x in (w - d, w + d):
                c, neg = ref.to_codes(np.ldexp(x, -s), fmt)
                ends.append(np.ldexp(ref.GRIDS[fmt][c] * np.where(neg, -1, 1), s))
        lo, hi = np.minimum.reduce(ends)[:, :K], np.maximum.reduce(ends)[:, :K]
        return (lo + hi) / 2, (hi - lo) / 2


class Loose:
    """Real numbers, a rounding's size in the bound: E4M3 keeps values to half a step, 2^-4 of
    them or 2^-10 of the scale, and cuts off those over 448 of up to 512 scales, an eighth; a
    bound that may double the scale doubles the small step."""
    @staticmethod
    def bf16(v, e):
        return v, e + 2.0 ** -8 * (np.abs(v) + e)

    @staticmethod
    def codes(v, e, fmt):
        assert fmt == "e4m3"
        R, K = v.shape
        a = np.hstack([np.abs(v) + e, np.zeros((R, dr.up32(K) - K))])
        top = np.repeat(a.reshape(R, -1, 32).max(-1), 32, axis=1)[:, :K]
        return v, e + (np.abs(v) + e) / 8 + top * 2.0 ** -17


def matmul(A, eA, B, eB):
    """A . B^T of (A, eA) and (B, eB)."""
    v = A @ B.T
    m = (np.abs(A) + eA) @ (np.abs(B) + eB).T
    return v, m - np.abs(A) @ np.abs(B).T + ACC * m


def act(v, e, kind):
    """act(z), act'(z) of z within e of v: slopes of at most 1.13, curvatures of at most 1.13."""
    h, slope, eh, es = dr.act(v, kind)
    return (h, 1.13 * e + eh), (slope, (1.13 * e if kind not in ("none", "relu") else np.where(np.abs(v) <= e, 1.0 * (e > 0), 0.0)) + es)


def forward(p, how, fmt):
    """p: x, w1, w2, b1, b2, norm_w, norm_b, act, eps -> every value of the forward pass."""
    r = {}
    y, r["mean"], r["rstd"], ey, r["emean"], r["erstd"] = dr.norm(p["x"], p["norm_w"], p["norm_b"], p["eps"])
    r["y"] = how.bf16(y, ey)
    z, ez = matmul(*how.codes(*r["y"], fmt), p["w1"], 0.0)
    z = z + p["b1"]
    r["z"] = z, ez + 2 * EPS24 * np.abs(z)
    r["h"] = act(*r["z"], p["act"])[0]
    d, ed = matmul(*how.codes(*r["h"], fmt), p["w2"], 0.0)
    d = d + p["b2"]
    out = d + p["x"]
    r["out"] = how.bf16(out, ed + 4 * EPS24 * (np.abs(d) + np.abs(out)))
    return r


def backward(p, dout, yt, z, how, fmt, fmt_grad):
    """Gradients from the kept yt (y^T as the product reads it) and z, each (v, e)."""
    T, K = dout.shape
    zero = np.zeros_like(dout)
    g = {}
    dh = how.bf16(*matmul(*how.codes(dout, zero, fmt_grad), p["w2t"], p.get("ew2t", 0.0)))
    (h, eh), (s, es) = act(*z, p["act"])
    dz = dh[0] * s
    edz = dh[1] * (np.abs(s) + es) + np.abs(dh[0]) * es + 2 * EPS24 * np.abs(dz)
    chain = (T / 32 + 64) * EPS24
    g["db1"] = dz.sum(0), edz.sum(0) + chain * (np.abs(dz) + edz).sum(0)
    g["db2"] = dout.sum(0), chain * np.abs(dout).sum(0)
    along = lambda v, e, f: how.codes(np.ascontiguousarray(v.T), np.ascontiguousarray(np.broadcast_to(e, v.shape).T), f)
    g["dw2"] = how.bf16(*matmul(*along(dout, zero, fmt_grad), *along(h, eh, fmt)))
    g["dw1"] = how.bf16(*matmul(*along(dz, edz, fmt_grad), *yt))
    dy, ey = how.bf16(*matmul(*how.codes(dz, edz, fmt_grad), p["w1t"], p.get("ew1t", 0.0)))
    mean, rstd, w = p["mean"], p["rstd"], p["norm_w"]
    dx, dw, db, edx, edw, edb = dr.norm_backward(p["x"], dy, mean, rstd, w, dout)
    xhat = np.abs((p["x"] - mean[:, None]) * rstd[:, None])
    eg = ey * np.abs(w)
    edx = 1.001 * edx + rstd[:, None] * (eg + eg.mean(1, keepdims=True) + xhat * (eg * xhat).mean(1, keepdims=True)) * 1.001
    # (the sums' own roundings: of dy's size, which ey can enlarge)
    chain = (T / 304 + 64) * EPS24
    g["dx"] = how.bf16(dx, edx)
    g["dnorm_w"] = dw, edw + (1 + 2 * chain) * (ey * xhat).sum(0)
    g["dnorm_b"] = db, edb + (1 + 2 * chain) * ey.sum(0)
    return g
