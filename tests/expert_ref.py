"""Plain 64-bit forms of the expert-layer operators, from their definitions,
and the layouts they use (numpy, CPU)."""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_grid():
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))


def e5m2_grid():
    c = np.arange(124)
    e, m = c >> 2, c & 3
    return np.where(e == 0, m * 2.0 ** -16, (4 + m) * 2.0 ** (e - 17.0))


GRIDS = {"e2m1": E2M1, "e4m3": e4m3_grid(), "e5m2": e5m2_grid()}
EMAX = {"e4m3": 8, "e5m2": 15}


def scale_exponent(amax, fmt):
    """s of one block's largest magnitude: the quantisers' rule."""
    if amax == 0:
        return 0
    m, e = np.frexp(amax)
    s = (e - 3 if m >= 0.75 else e - 4) if fmt == "e2m1" else e - 1 - EMAX[fmt]
    return int(min(127, max(-127, s)))


def to_codes(y, fmt):
    """Magnitude codes and signs of scaled values: nearest, ties to the even code, saturating."""
    grid = GRIDS[fmt]
    a = np.minimum(np.abs(y), grid[-1])
    hi = np.minimum(np.searchsorted(grid, a), len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    down, up = a - grid[lo], grid[hi] - a
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return code, np.signbit(y)


def quantise(x, fmt):
    """x [rows, K] float64 -> codes as stored [rows, K / 2 or K], scales [rows, K / 32]."""
    rows, K = x.shape
    b = x.reshape(rows, K // 32, 32)
    amax = np.abs(b).max(-1)
    s = np.vectorize(lambda v: scale_exponent(v, fmt), otypes=[int])(amax)
    code, neg = to_codes(np.ldexp(b, -s[..., None]), fmt)
    code, neg = code.reshape(rows, K), neg.reshape(rows, K)
    if fmt == "e2m1":
        c = (code | neg << 3).astype(np.uint8)
        return c[:, 0::2] | c[:, 1::2] << 4, (s + 127).astype(np.uint8)
    return (code | neg.astype(int) << 7).astype(np.uint8), (s + 127).astype(np.uint8)


def values(codes, scales, fmt):
    """Stored codes and E8M0 scales -> float64 values [rows, K] (NaN scales give NaN)."""
    codes = np.asarray(codes)
    if fmt == "e2m1":
        c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
        v = E2M1[c & 7] * np.where(c & 8, -1.0, 1.0)
    elif fmt in PADDED:
        v = padded_values(codes, fmt)
    else:
        mag = codes & 0x7F
        grid = np.full(128, np.nan)
        grid[:len(GRIDS[fmt])] = GRIDS[fmt]
        v = grid[mag] * np.where(codes & 0x80, -1.0, 1.0)
    p = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(int) - 127))
    return v * np.repeat(p, 32, axis=-1)


# Sub-byte formats, 16 codes packed at the start of every 16 bytes: exponent and mantissa bits.
PADDED = {"e2m3": (2, 3), "e3m2": (3, 2), "e2m1 padded": (2, 1)}


def padded_values(codes, fmt):
    ebits, mbits = PADDED[fmt]
    width, bias = 1 + ebits + mbits, 2 ** (ebits - 1) - 1
    bits = np.unpackbits(codes.reshape(*codes.shape[:-1], -1, 16), axis=-1, bitorder="little")
    c = (bits[..., :16 * width].reshape(*bits.shape[:-1], 16, width).astype(int) << np.arange(width)).sum(-1)
    e, m = c >> mbits & 2 ** ebits - 1, c & 2 ** mbits - 1
    v = np.where(e == 0, np.ldexp(1.0 * m, 1 - bias - mbits), np.ldexp(1.0 * m + 2 ** mbits, e - bias - mbits))
    return (np.where(c >> width - 1, -1.0, 1.0) * v).reshape(codes.shape)


def grouping(ids, E):
    """ids [T, k] -> offsets, row_token, slot_row."""
    T, k = ids.shape
    offsets, row_token, slot_row = [0], [], np.full((T, k), -1, np.int32)
    for e in range(E):
        for t in range(T):
            for j in range(k):
                if ids[t, j] == e:
                    slot_row[t, j] = len(row_token)
                    row_token.append(t)
        offsets.append(len(row_token))
    full = np.full(T * k, -1, np.int32)
    full[:len(row_token)] = row_token
    return np.array(offsets, np.int32), full, slot_row


def route(logits, k, mode, mask=None):
    """logits float64 [T, E] -> ids, gates (mode 0 softmax of the picked, 1 of all, 2 sigmoid)."""
    T, E = logits.shape
    ids, gates = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t in range(T):
        x = np.where(np.isnan(logits[t]), -np.inf, logits[t])
        if mask is not None and not mask[t]:
            continue
        pick = [e for e in sorted(range(E), key=lambda e: (-x[e], e)) if x[e] > -np.inf][:k]
        if not pick:
            continue
        ids[t, :len(pick)] = pick
        v, top = x[pick], x[pick[0]]
        over = x if mode == 1 else v
        with np.errstate(invalid="ignore"):
            ex = lambda z: np.where(z == top, 1.0, np.exp(z - top))
            gates[t, :len(pick)] = 1 / (1 + np.exp(-v)) if mode == 2 else ex(v) / ex(over).sum()
    return ids, gates


def route_many(logits, k, mode, mask=None):
    """route() and grouping() without loops over the tokens, for many of them."""
    x = np.where(np.isnan(logits), -np.inf, logits)
    if mask is not None:
        x = np.where(mask[:, None] != 0, x, -np.inf)
    order = np.argsort(-x, axis=1, kind="stable")[:, :k]
    v = np.take_along_axis(x, order, 1)
    fine = v > -np.inf
    top = np.where(fine[:, :1], v[:, :1], 0)
    with np.errstate(invalid="ignore", over="ignore"):
        ex = lambda z: np.where(z == top, 1.0, np.where(z > -np.inf, np.exp(z - top), 0.0))
        gates = 1 / (1 + np.exp(-v)) if mode == 2 else ex(v) / np.maximum((ex(x) if mode == 1 else ex(v)).sum(1, keepdims=True), 1)
    ids = np.where(fine, order, -1).astype(np.int32)
    E, flat = x.shape[1], np.where(ids < 0, x.shape[1], ids).reshape(-1)
    by = np.argsort(flat, kind="stable")
    offsets = np.searchsorted(flat[by], np.arange(E + 1)).astype(np.int32)
    place = np.empty(flat.size, np.int32)
    place[by] = np.arange(flat.size)
    rows = np.where(np.arange(flat.size) < offsets[E], by // k, -1).astype(np.int32)
    return ids, np.where(fine, gates, 0), offsets, rows, np.where(flat < E, place, -1).reshape(ids.shape)


def sf_groups(K):
    return 2 * (-(-K // 256))


def scale_places(offsets, K):
    """Byte of the grouped layout of every (row, 32-block): int64 [rows, K / 32]."""
    out = []
    for e in range(len(offsets) - 1):
        for r in range(offsets[e], offsets[e + 1]):
            i = r - offsets[e]
            block, i = offsets[e] // 128 + e + i // 128, i % 128
            b = np.arange(K // 32)
            out.append((block * sf_groups(K) + b // 4) * 512 + 16 * (i % 32) + 4 * (i // 32) + b % 4)
    return np.array(out, np.int64).reshape(-1, K // 32)


def grouped_scales(S, offsets, K, rows, fill=127):
    """Row-major scales [>= offsets[-1], K / 32] -> the grouped layout for `rows` rows."""
    flat = np.full((rows // 128 + len(offsets) - 1) * sf_groups(K) * 512, fill, np.uint8)
    at = scale_places(offsets, K)
    flat[at] = S[:len(at)]
    # The partner of a last odd block has to be finite.
    if (K // 32) % 2 and len(at):
        flat[at[:, -1] + 1] = 127
    return flat


def relaid(S, K):
    """Weight scales [rows, K / 32] -> atoms of 128 rows x 4 blocks, padded with 1.0."""
    rows = S.shape[0]
    rb, groups = 2 * (-(-rows // 256)), sf_groups(K)
    full = np.full((rb * 128, groups * 4), 127, np.uint8)
    full[:rows, :K // 32] = S
    return full.reshape(rb, 4, 32, groups, 4).transpose(0, 3, 2, 1, 4).copy().reshape(-1)


def product(A, B, offsets):
    """(A[r] . B[e]^T, sum |a b|) for the rows of each group; A [R, K], B [E, N, K]."""
    D = np.zeros((A.shape[0], B.shape[1]))
    S = np.zeros_like(D)
    for e in range(len(offsets) - 1):
        a = A[offsets[e]:offsets[e + 1]]
        D[offsets[e]:offsets[e + 1]] = a @ B[e].T
        S[offsets[e]:offsets[e + 1]] = np.abs(a) @ np.abs(B[e]).T
    return D, S


def combine(Y, slot_row, gates, resid, w_post, w_pre, res_scale, out_scale, eps):
    """(h, n, magnitude sums that bound their fp32 error)."""
    T, k = slot_row.shape
    b, m = np.zeros((T, Y.shape[1])), np.zeros((T, Y.shape[1]))
    for t in range(T):
        for j in range(k):
            if slot_row[t, j] >= 0:
                b[t] += gates[t, j] * Y[slot_row[t, j]]
                m[t] += np.abs(gates[t, j] * Y[slot_row[t, j]])
    if w_post is not None:
        r = 1 / np.sqrt((b * b).mean(1, keepdims=True) + eps)
        b, m = b * r * w_post, m * r * np.abs(w_post)
    h = out_scale * b + (0 if resid is None else res_scale * resid)
    m = np.abs(out_scale) * m + (0 if resid is None else np.abs(res_scale * resid))
    r = 1 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    w = 1.0 if w_pre is None else w_pre
    return h, h * r * w, m, m * r * np.abs(w)
