"""Cases that time the mixture-of-experts operators on block-scaled operands.

Six operators, each with a plain form in elementary torch operations (32-bit
arithmetic, one rounding at the end) and the library's own calls:

  route     logits [T, E] -> the k largest experts of each token, their gates
            and the grouping of the (token, slot) rows by expert
  quantize  bf16 rows -> MXFP8 rows copied to their places in the grouping,
            scales in the grouped 128-row-block layout
  gemm      D[r] = A[r] . B[e]^T for every row r of group e (MXFP4)
  swiglu    H[r] = quantise(silu(A[r] . Bg[e]^T) * (A[r] . Bu[e]^T)) (MXFP8)
  ffn       a routed block on MXFP4: quantise, both products, combine, norm
  combine   the gated sum of a token's expert rows, normalised, added to the
            residual stream, and the norm in front of the next block

What is held in 8 bits is returned as the float8 values it stands for (codes
as E4M3, scales as E8M0); the packed 4-bit rows stay inside `ffn`.
"""
import math

import numpy as np
import torch

own = False

BF16, FP32 = 0, 1                      # logits' type
GATE_TOPK, GATE_ALL, GATE_SIGMOID = 0, 1, 2
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
WORKSPACE = 64 << 20                   # more than any split of the grouped products needs


def listed():
    return [
        # One decoding step of sixteen sequences: pure latency.
        dict(name="route decode", op="route", T=16, E=128, k=8, dtype="bf16", mode=GATE_TOPK, masked=0.0),
        # A long prefill with padding tokens among it, the gates not renormalised.
        dict(name="route prefill", op="route", T=32768, E=256, k=8, dtype="fp32", mode=GATE_ALL, masked=0.06),
        # A small batch's rows on the way to their experts.
        dict(name="quantize batch", op="quantize", T=64, E=32, k=4, K=2048, masked=0.0),
        # A prefill's rows, each copied to four experts.
        dict(name="quantize prefill", op="quantize", T=8192, E=64, k=4, K=8192, masked=0.03),
        # Decoding: a few rows for each expert that has any, the weights' bytes rule.
        dict(name="gemm decode", op="gemm", T=4, E=64, k=8, N=4096, K=4096, skew=0.5),
        # A prefill's down projection, groups of every size, N no multiple of a tile.
        dict(name="gemm prefill", op="gemm", T=8192, E=32, k=4, N=4000, K=2048, skew=0.6),
        # A mid-sized batch on byte operands.
        dict(name="swiglu batch", op="swiglu", T=512, E=16, k=4, F=1024, K=2048, skew=0.5),
        # A prefill's gate and up projections on byte operands.
        dict(name="swiglu prefill", op="swiglu", T=4096, E=32, k=4, F=2048, K=4096, skew=0.6),
        # One token through its eight experts.
        dict(name="ffn decode", op="ffn", T=1, E=64, k=8, F=2048, K=4096, skew=0.0, masked=0.0),
        # A prefill through the whole block, some of its tokens padding.
        dict(name="ffn prefill", op="ffn", T=4096, E=32, k=4, F=2048, K=4096, skew=0.6, masked=0.05),
        # Joining a decoding batch's expert rows.
        dict(name="combine decode", op="combine", T=8, k=8, N=7168, post=False, masked=0.0),
        # Joining a prefill's, with a norm on either side.
        dict(name="combine prefill", op="combine", T=8192, k=4, N=8192, post=True, masked=0.03),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def of32(lo, hi):
        return 32 * log(lo // 32, hi // 32)

    op = rng.choice(["route", "quantize", "gemm", "gemm", "swiglu", "ffn", "ffn", "combine"])
    masked = rng.choice([0.0, 0.02, 0.1])
    skew = rng.choice([0.0, 0.4, 0.8])
    if op == "route":
        E = log(4, 512)
        return dict(op=op, T=log(1, 32768), E=E, k=min(E, rng.randint(1, 10)), dtype=rng.choice(["bf16", "fp32"]),
                    mode=rng.choice([GATE_TOPK, GATE_ALL, GATE_SIGMOID]), masked=masked)
    if op == "quantize":
        return dict(op=op, T=log(1, 8192), E=log(8, 128), k=rng.randint(1, 4), K=of32(256, 8192), masked=masked)
    if op == "combine":
        return dict(op=op, T=log(1, 8192), k=rng.randint(1, 4), N=log(256, 8192), post=rng.random() < 0.5, masked=masked)
    E = log(8, 64)
    k = rng.randint(1, 4)
    T = log(1, 4096)
    K = of32(512, 4096)
    if op == "gemm":
        n = log(256, 4096)
        return dict(op=op, T=T, E=E, k=k, N=n if rng.random() < 0.25 else -(-n // 8) * 8, K=K, skew=skew)
    if op == "swiglu":
        return dict(op=op, T=T, E=E, k=k, F=of32(256, 2048), K=K, skew=skew)
    return dict(op=op, T=T, E=E, k=k, F=of32(256, 2048), K=K, skew=skew, masked=masked)


# ------------------------------------------------------------------ the routing --


def routing(case):
    """Which experts each token takes: numpy ids [T, k], -1 where it takes none.
    A matter of the case alone, so that the work is too."""
    T, E, k = case["T"], case["E"], case["k"]
    r = np.random.RandomState(T * 7 + E * 131 + k)
    bias = -case.get("skew", 0.3) * np.log(np.arange(1, E + 1))
    r.shuffle(bias)
    score = r.gumbel(size=(T, E)).astype(np.float32) + bias.astype(np.float32)
    ids = np.argsort(-score, axis=1, kind="stable")[:, :k].astype(np.int32)
    if case.get("masked"):
        ids[r.uniform(size=T) < case["masked"]] = -1
    return ids


def grouping(ids, E):
    """ids [T, k] -> offsets [E + 1], row_token [T k], slot_row [T, k], as torch tensors like ids."""
    T, k = ids.shape
    flat = torch.where(ids < 0, E, ids).reshape(-1).long()
    order = torch.argsort(flat, stable=True)
    count = torch.searchsorted(flat[order], torch.arange(E + 1, device=ids.device))
    total = count[E]
    place = torch.empty_like(flat)
    place[order] = torch.arange(T * k, device=ids.device)
    slot_row = torch.where(flat < E, place, -1).reshape(T, k)
    row_token = torch.where(torch.arange(T * k, device=ids.device) < total, order // k, -1)
    return count.int(), row_token.int(), slot_row.int()


def counts(case):
    ids = routing(case)
    return np.bincount(ids[ids >= 0].reshape(-1), minlength=case["E"])


# ------------------------------------------------------------------ the layouts --


def blocks_of(K):
    return 2 * (-(-K // 256))          # 128-row blocks of scales hold this many 512-byte atoms


def scale_bytes(R, E, K):
    return (R // 128 + E) * blocks_of(K) * 512


def scale_places(offsets, R, K):
    """Where the scale of (grouped row, 32-block) sits in the grouped layout: [R, K / 32]; rows past the groups get -1."""
    dev = offsets.device
    r = torch.arange(R, device=dev)
    e = torch.searchsorted(offsets[1:].long(), r, right=True).clamp(max=offsets.numel() - 2)
    start = offsets.long()[e]
    local = r - start
    rb = start // 128 + e + local // 128
    i = local % 128
    b = torch.arange(K // 32, device=dev)
    at = (rb[:, None] * blocks_of(K) + b // 4) * 512 + (16 * (i % 32) + 4 * (i // 32))[:, None] + b % 4
    return torch.where((r < offsets[-1])[:, None], at, -1)


def relaid(S):
    """Weights' scales [..., rows, K / 32] -> one block layout per matrix (rows padded to 256, K to 256, with 1.0)."""
    *lead, rows, kb = S.shape
    groups = blocks_of(kb * 32)
    rb = 2 * (-(-rows // 256))
    full = torch.full((*lead, rb * 128, groups * 4), 127, dtype=torch.uint8, device=S.device)
    full[..., :rows, :kb] = S
    full = full.reshape(*lead, rb, 4, 32, groups, 4)          # row 32 j + i, block 4 g + b
    n = len(lead)
    return full.permute(*range(n), n, n + 3, n + 2, n + 1, n + 4).contiguous()


# ------------------------------------------------------------------ the inputs --


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = "cuda"

    def normal(*shape, scale=1.0, dtype=torch.bfloat16):
        out = torch.empty(shape, dtype=dtype, device=dev)
        if out.dim() > 2 or dtype == torch.float32:
            return out.normal_(0, scale, generator=g)
        return torch.randn(shape, device=dev, generator=g).mul_(scale).to(dtype)

    def activations(rows, n):
        """Rows as a norm leaves them: unit scale, a few channels much larger."""
        x = torch.randn((rows, n), device=dev, generator=g)
        x *= 1 + 7 * (torch.rand((1, n), device=dev, generator=g) < 0.01)
        return x.to(torch.bfloat16)

    def weights4(*shape):
        """Packed E2M1 rows [..., K / 2] of normal weights, scales [..., K / 32]."""
        *lead, K = shape
        q = torch.empty((*lead, K // 2), dtype=torch.uint8, device=dev)
        limits = torch.tensor([(a + b) / 2 for a, b in zip(E2M1, E2M1[1:])], device=dev)
        for part in q.view(-1, *q.shape[-2:]):
            x = torch.randn((*part.shape, 2), device=dev, generator=g).mul_(2.5)
            c = torch.bucketize(x.abs(), limits).to(torch.uint8) | (x < 0).to(torch.uint8) << 3
            part.copy_(c[..., 0] | c[..., 1] << 4)
        s = torch.randint(118, 121, (*lead, K // 32), dtype=torch.uint8, device=dev, generator=g)
        return q, s

    def weights8(*shape):
        *lead, K = shape
        q = torch.empty(shape, dtype=torch.uint8, device=dev)
        for part in q.view(-1, *q.shape[-2:]):
            x = torch.randn(part.shape, device=dev, generator=g).mul_(100).clamp_(-448, 448)
            part.copy_(x.to(torch.float8_e4m3fn).view(torch.uint8))
        s = torch.randint(114, 117, (*lead, K // 32), dtype=torch.uint8, device=dev, generator=g)
        return q, s

    def routed(s):
        ids = torch.from_numpy(routing(case)).to(dev)
        s["ids"] = ids
        s["offsets"], s["row_token"], s["slot_row"] = grouping(ids, case["E"])
        s["gates"] = torch.rand(ids.shape, device=dev, generator=g).mul_(ids >= 0) * (2 / case["k"])
        s["cap"] = max(1, int(counts(case).max()))

    op, T = case["op"], case["T"]
    k = case["k"]
    s = {"case": case}
    if op == "route":
        E = case["E"]
        x = torch.randn((T, E), device=dev, generator=g).mul_(1.5)
        x -= 0.7 * torch.rand((1, E), device=dev, generator=g)
        s["logits"] = x.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
        s["mask"] = (torch.rand((T,), device=dev, generator=g) >= case["masked"]) if case["masked"] else None
        i32 = dict(dtype=torch.int32, device=dev)
        s["out"] = dict(ids=torch.empty((T, k), **i32), gates=torch.empty((T, k), device=dev), offsets=torch.empty(E + 1, **i32),
                        row_token=torch.empty(T * k, **i32), slot_row=torch.empty((T, k), **i32))
        s["workspace"] = torch.empty(WORKSPACE, dtype=torch.uint8, device=dev)
        return s
    if op == "quantize":
        R, K = T * k, case["K"]
        routed(s)
        s["x"] = activations(T, K)
        s["codes"] = torch.zeros((R, K), dtype=torch.uint8, device=dev)
        s["scales"] = torch.full((scale_bytes(R, case["E"], K),), 127, dtype=torch.uint8, device=dev)
        return s
    if op == "combine":
        N = case["N"]
        r = np.random.RandomState(T + N)
        rows = torch.from_numpy(r.permutation(T * k).astype(np.int32)).to(dev).reshape(T, k)
        if case["masked"]:
            rows[torch.from_numpy(r.uniform(size=T) < case["masked"]).to(dev)] = -1
        s["slot_row"] = rows.contiguous()
        s["gates"] = torch.rand((T, k), device=dev, generator=g) / k
        s["y"] = torch.randn((T * k, N), device=dev, generator=g).to(torch.bfloat16)
        s["resid"] = torch.randn((T, N), device=dev, generator=g).mul_(3).to(torch.bfloat16)
        s["w_post"] = normal(N, scale=0.2) + 1 if case["post"] else None
        s["w_pre"] = normal(N, scale=0.2) + 1
        s["h"] = torch.empty((T, N), dtype=torch.bfloat16, device=dev)
        s["n"] = torch.empty((T, N), dtype=torch.bfloat16, device=dev)
        return s
    E, K, R = case["E"], case["K"], T * k
    routed(s)
    s["workspace"] = torch.empty(WORKSPACE, dtype=torch.uint8, device=dev)
    if op == "gemm":
        s["A"], s["SA"] = weights4(1, R, K)
        s["A"], s["SA"] = s["A"][0], s["SA"][0] + 7
        s["B"], s["SB"] = weights4(E, case["N"], K)
        s["D"] = torch.zeros((R, case["N"]), dtype=torch.bfloat16, device=dev)
    elif op == "swiglu":
        s["A"], s["SA"] = weights8(1, R, K)
        s["A"], s["SA"] = s["A"][0], s["SA"][0] + 5
        s["B"], s["SB"] = weights8(E, 2, case["F"], K)
        s["codes"] = torch.zeros((R, case["F"]), dtype=torch.uint8, device=dev)
        s["scales"] = torch.full((scale_bytes(R, E, case["F"]),), 127, dtype=torch.uint8, device=dev)
    else:
        F = case["F"]
        s["x"] = activations(T, K)
        s["resid"] = torch.randn((T, K), device=dev, generator=g).mul_(0.2).to(torch.bfloat16)
        s["w_pre"] = normal(K, scale=0.2) + 1
        s["B1"], s["S1"] = weights4(E, 2, F, K)
        s["B2"], s["S2"] = weights4(E, K, F)
        s["S1r"], s["S2r"] = relaid(s["S1"]), relaid(s["S2"])
        s["h"] = torch.empty((T, K), dtype=torch.bfloat16, device=dev)
        s["n"] = torch.empty((T, K), dtype=torch.bfloat16, device=dev)
        s["arena"] = torch.empty(WORKSPACE + R * (2 * K + K // 2 + F // 2) + scale_bytes(R, E, K) + scale_bytes(R, E, F) + 4096,
                                 dtype=torch.uint8, device=dev)
        return s
    # The rows' scales in the grouped layout, the weights' in the block layout: both laid out once.
    at = scale_places(s["offsets"], R, K)
    lay = torch.full((scale_bytes(R, E, K),), 127, dtype=torch.uint8, device=dev)
    lay[at[at >= 0]] = s["SA"][at >= 0]
    s["SAr"], s["SBr"] = lay, relaid(s["SB"])
    return s


# ------------------------------------------------------------------ the plain forms --


def two_to(s):
    """2^s for whole s, exactly (a power by bits: pow() may be a unit off), in 64 bits."""
    return ((s.long() + 1023) << 52).view(torch.float64)


def values4(q, s, dtype=torch.float32):
    """Packed E2M1 [..., K / 2] and E8M0 [..., K / 32] -> values [..., K]."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=dtype, device=q.device)
    v = torch.stack((lut[(q & 15).int()], lut[(q >> 4).int()]), -1).flatten(-2)
    return (v.unflatten(-1, (-1, 32)) * two_to(s.int() - 127).to(dtype)[..., None]).flatten(-2)


def values8(q, s, dtype=torch.float32):
    v = q.view(torch.float8_e4m3fn).to(dtype)
    return (v.unflatten(-1, (-1, 32)) * two_to(s.int() - 127).to(dtype)[..., None]).flatten(-2)


def exponent(amax, fmt):
    """The block's scale 2^s: MXFP4 the largest with 6 2^s <= amax, E4M3 floor(log2 amax) - 8; 0 for zeros."""
    m, e = torch.frexp(amax)
    s = e - torch.where(m >= 0.75, 3, 4) if fmt == 4 else e - 9
    return torch.where(amax == 0, 0, s.clamp(-127, 127))


def quantised(x, fmt):
    """x [..., K] -> (values on the format's grid before scaling, s [..., K / 32])."""
    x = x.unflatten(-1, (-1, 32))
    s = exponent(x.abs().amax(-1), fmt)
    y = x * two_to(-s).to(x.dtype)[..., None]
    if fmt == 8:
        return y.clamp(-448, 448).to(torch.float8_e4m3fn).flatten(-2), s
    a = y.abs().clamp(max=6)
    a = torch.where(a < 2, torch.round(a * 2) / 2, torch.where(a < 4, torch.round(a), torch.round(a / 2) * 2))
    return torch.copysign(a, y).flatten(-2), s


def by_group(A, offsets, cap):
    """Rows [R, K] -> [E, cap, K], groups padded with zeros, and where each row sits in it."""
    E, R = offsets.numel() - 1, A.shape[0]
    r = torch.arange(R, device=A.device)
    e = torch.searchsorted(offsets[1:].long(), r, right=True)
    at = torch.where(r < offsets[-1], e.clamp(max=E - 1) * cap + r - offsets.long()[e.clamp(max=E - 1)], E * cap)
    G = torch.zeros((E * cap + 1, A.shape[1]), dtype=A.dtype, device=A.device)
    G[at] = A
    return G[:-1].view(E, cap, -1), at


def product(A, B, offsets, cap):
    """Rows A [R, K] and B [E, N, K] -> [R, N]; rows of no group are zero."""
    G, at = by_group(A, offsets, cap)
    D = torch.bmm(G, B.transpose(1, 2)).flatten(0, 1)
    return torch.cat((D, torch.zeros_like(D[:1])))[at]


def rms(x, w, eps):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w


def joined(y, slot_row, gates, resid, w_post, w_pre, eps):
    """The gated sum of y's rows, the residual stream after it, and its norm, in y's type."""
    picked = torch.where((slot_row >= 0)[..., None], y[slot_row.clamp(min=0).long()], 0)
    b = (picked * torch.where(slot_row >= 0, gates, 0)[..., None]).sum(1)
    if w_post is not None:
        b = rms(b, w_post, eps)
    h = resid + 0.5 * b
    return h, rms(h, w_pre, eps)


EPS = 1e-6


def plain(s):
    case = s["case"]
    op, k = case["op"], case["k"]
    if op == "route":
        E = case["E"]
        x = s["logits"].float()
        x = torch.where(torch.isnan(x), -math.inf, x)
        if s["mask"] is not None:
            x = torch.where(s["mask"][:, None], x, -math.inf)
        v, ids = torch.sort(x, dim=1, descending=True, stable=True)
        v, ids = v[:, :k], ids[:, :k]
        fine = v > -math.inf
        if case["mode"] == GATE_SIGMOID:
            gates = 1 / (1 + torch.exp(-v))
        else:
            top = torch.where(fine[:, :1], v[:, :1], 0)
            e = torch.exp((x if case["mode"] == GATE_ALL else v) - top)
            gates = torch.exp(v - top) / torch.where(fine[:, :1], e.sum(1, keepdim=True), 1)
        ids = torch.where(fine, ids, -1).int()
        offsets, row_token, slot_row = grouping(ids, E)
        return dict(ids=ids, gates=torch.where(fine, gates, 0), offsets=offsets, row_token=row_token, slot_row=slot_row)
    if op == "quantize":
        R, K = case["T"] * k, case["K"]
        q, e = quantised(s["x"].float(), 8)
        row = s["slot_row"].reshape(-1).long()
        took = row >= 0
        codes = torch.zeros((R, K), dtype=torch.uint8, device=row.device)
        codes[row[took]] = q.view(torch.uint8).repeat_interleave(k, 0)[took]
        at = scale_places(s["offsets"], R, K)
        scales = torch.full_like(s["scales"], 127)
        scales[at[row[took]]] = (e + 127).to(torch.uint8).repeat_interleave(k, 0)[took]
        return dict(codes=codes.view(torch.float8_e4m3fn), scales=scales.view(torch.float8_e8m0fnu))
    if op == "gemm":
        return product(values4(s["A"], s["SA"]), values4(s["B"], s["SB"]), s["offsets"], s["cap"]).to(torch.bfloat16)
    if op == "swiglu":
        R, F = s["codes"].shape
        gu = product(values8(s["A"], s["SA"]), values8(s["B"], s["SB"]).flatten(1, 2), s["offsets"], s["cap"])
        g, u = gu[:, :F], gu[:, F:]
        q, e = quantised(g / (1 + torch.exp(-g)) * u, 8)
        at = scale_places(s["offsets"], R, F)
        scales = torch.full_like(s["scales"], 127)
        scales[at[at >= 0]] = (e + 127).to(torch.uint8)[at >= 0]
        return dict(codes=q, scales=scales.view(torch.float8_e8m0fnu))
    if op == "ffn":
        T, F, K = case["T"], case["F"], case["K"]
        R = T * k
        q, e = quantised(s["x"].float(), 4)
        x = (q.unflatten(-1, (-1, 32)) * two_to(e).to(q.dtype)[..., None]).flatten(-2)
        A = torch.where((s["row_token"] >= 0)[:, None], x[s["row_token"].clamp(min=0).long()], 0)
        gu = product(A, values4(s["B1"], s["S1"]).flatten(1, 2), s["offsets"], s["cap"])
        g, u = gu[:, :F], gu[:, F:]
        q, e = quantised(g / (1 + torch.exp(-g)) * u, 4)
        H = (q.unflatten(-1, (-1, 32)) * two_to(e).to(q.dtype)[..., None]).flatten(-2)
        y = product(H, values4(s["B2"], s["S2"]), s["offsets"], s["cap"])
        h, n = joined(y, s["slot_row"], s["gates"], s["resid"].float(), None, s["w_pre"].float(), EPS)
        return dict(h=h.to(torch.bfloat16), n=n.to(torch.bfloat16))
    w_post = None if s["w_post"] is None else s["w_post"].float()
    h, n = joined(s["y"].float(), s["slot_row"], s["gates"], s["resid"].float(), w_post, s["w_pre"].float(), EPS)
    return dict(h=h.to(torch.bfloat16), n=n.to(torch.bfloat16))


# ------------------------------------------------------------------ the library's calls --


def library(s):
    import block_scaled_mxfp4_gb300 as mx
    case = s["case"]
    op, T, k = case["op"], case["T"], case["k"]
    if op == "route":
        o, x, ws = s["out"], s["logits"], s["workspace"]
        mx.mxfp4_moe_route(o["ids"], o["gates"], o["offsets"], o["row_token"], o["slot_row"], x, x.stride(0),
                           mx.MXFP4_LOGITS_BF16 if case["dtype"] == "bf16" else mx.MXFP4_LOGITS_FP32, s["mask"], T, case["E"], k,
                           (mx.MXFP4_GATE_TOPK, mx.MXFP4_GATE_ALL, mx.MXFP4_GATE_SIGMOID)[case["mode"]], 1.0, ws, ws.numel())
        return o
    if op == "quantize":
        K = case["K"]
        mx.mxfp8_group_quantize(s["codes"], K, s["scales"], s["x"], K, T, K, s["slot_row"], s["ids"], k, s["offsets"], case["E"],
                                T * k, mx.MXFP8_E4M3)
        return dict(codes=s["codes"].view(torch.float8_e4m3fn), scales=s["scales"].view(torch.float8_e8m0fnu))
    if op == "combine":
        N = case["N"]
        mx.mxfp4_moe_combine(s["h"], N, s["n"], N, s["y"], N, T * k, s["slot_row"], s["gates"], k, s["resid"], N, s["w_post"],
                             s["w_pre"], 1.0, 0.5, EPS, T, N)
        return dict(h=s["h"], n=s["n"])
    E, K, R = case["E"], case["K"], T * k
    if op == "gemm":
        N, ws = case["N"], s["workspace"]
        mx.mxfp4_grouped_gemm(s["D"], N, s["A"], K, s["SAr"], s["B"], K, N * K, s["SBr"], s["offsets"], E, R, N, K, 1.0, ws, ws.numel())
        return s["D"]
    if op == "swiglu":
        F, ws = case["F"], s["workspace"]
        mx.mxfp8_grouped_swiglu(s["codes"], F, s["scales"], s["A"], K, s["SAr"], s["B"], K, 2 * F * K, s["SBr"], s["offsets"], E, R, F, K,
                                mx.MXFP8_E4M3, mx.MXFP8_E4M3, mx.MXFP8_E4M3, 1.0, ws, ws.numel())
        return dict(codes=s["codes"].view(torch.float8_e4m3fn), scales=s["scales"].view(torch.float8_e8m0fnu))
    F, ws = case["F"], s["arena"]
    mx.mxfp4_moe_ffn(s["h"], K, s["n"], K, s["x"], K, s["ids"], s["gates"], s["offsets"], s["slot_row"], T, E, k, K, F, s["B1"], K, s["S1r"],
                     s["B2"], F, s["S2r"], s["resid"], K, None, s["w_pre"], 1.0, 0.5, EPS, ws, ws.numel())
    return dict(h=s["h"], n=s["n"])


def run(state):
    return library(state) if own else plain(state)


# ------------------------------------------------------------------ the work --


def work(case):
    op, T, k = case["op"], case["T"], case["k"]
    if op == "route":
        size = 2 if case["dtype"] == "bf16" else 4
        return dict(bytes=T * case["E"] * size + T * k * 16 + 4 * (case["E"] + 1), flops=T * case["E"])
    if op == "combine":
        N = case["N"]
        return dict(bytes=T * k * N * 2 + T * k * 8 + 3 * T * N * 2, flops=2 * T * k * N + 6 * T * N)
    c = counts(case)
    rows, active, K = int(c.sum()), int((c > 0).sum()), case["K"]
    if op == "quantize":
        return dict(bytes=T * K * 2 + rows * (K + K // 32) + 8 * T * k, flops=3 * T * K)
    if op == "gemm":
        N = case["N"]
        return dict(bytes=(rows + active * N) * (K // 2 + K // 32) + rows * N * 2, flops=2 * rows * N * K)
    F = case["F"]
    if op == "swiglu":
        return dict(bytes=(rows + active * 2 * F) * (K + K // 32) + rows * (F + F // 32), flops=4 * rows * F * K)
    weights = active * (2 * F * (K // 2 + K // 32) + K * (F // 2 + F // 32))
    return dict(bytes=weights + T * K * 2 * 4 + T * k * 12, flops=6 * rows * F * K)


# ------------------------------------------------------------------ 64 bits --


def nearest(x, grid):
    """x rounded to the nearest value of an ascending grid of magnitudes (even places on ties), its sign kept."""
    a = x.abs().clamp(max=float(grid[-1]))
    hi = torch.searchsorted(grid, a.contiguous()).clamp(max=grid.numel() - 1)
    lo = (hi - 1).clamp(min=0)
    down, up = a - grid[lo], grid[hi] - a
    take = (up < down) | ((up == down) & (hi % 2 == 0))
    return torch.where(take, grid[hi], grid[lo]) * torch.where(x < 0, -1.0, 1.0)


def quantised64(x, fmt):
    """(grid values, scales as powers of two) of 64-bit rows, from the definition."""
    x = x.reshape(*x.shape[:-1], -1, 32)
    amax = x.abs().amax(-1)
    ref = amax / 6 if fmt == 4 else amax / 256
    powers = torch.tensor([2.0 ** i for i in range(-127, 128)], dtype=torch.float64, device=x.device)
    scale = powers[(torch.searchsorted(powers, ref, right=True) - 1).clamp(min=0)]     # the largest that is not above
    scale = torch.where(amax > 0, scale, 1.0)
    if fmt == 4:
        grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    else:
        grid = torch.arange(127, dtype=torch.uint8, device=x.device).view(torch.float8_e4m3fn).double()
    q = nearest(x / scale[..., None], grid)
    return q.reshape(*q.shape[:-2], -1), scale


def exact(case, seed):
    s = prepare(case, seed)
    op, T, k = case["op"], case["T"], case["k"]
    if op == "route":
        x = s["logits"].double()
        if s["mask"] is not None:
            x[~s["mask"]] = -math.inf
        v = torch.topk(x, k, dim=1).values
        if case["mode"] == GATE_SIGMOID:
            gates = torch.sigmoid(v)
        elif case["mode"] == GATE_ALL:
            gates = torch.exp(v - torch.logsumexp(x, 1, keepdim=True))
        else:
            gates = torch.softmax(v, 1)
        return dict(ids=None, gates=torch.nan_to_num(gates), offsets=None, row_token=None, slot_row=None)
    off = s["offsets"].tolist() if "offsets" in s else None

    def one_by_one(f, out, E):
        for e in range(E):
            a, b = off[e], off[e + 1]
            if b > a:
                out[a:b] = f(e, a, b)
        return out

    def placed(scales, S, K):
        """S [R, K / 32] written into the grouped layout, a group at a time."""
        groups = blocks_of(K)
        flat = torch.ones(scales.numel(), dtype=torch.float64, device=S.device)
        view = flat.view(-1, groups, 32, 4, 4)                       # block, atom, i, j, b
        for e in range(case["E"]):
            for a in range(off[e], off[e + 1], 128):
                n = min(128, off[e + 1] - a)
                part = torch.ones((128, groups * 4), dtype=torch.float64, device=S.device)
                part[:n, :K // 32] = S[a:a + n]
                view[off[e] // 128 + e + (a - off[e]) // 128] = part.view(4, 32, groups, 4).permute(2, 1, 0, 3)
        return flat

    if op == "quantize":
        R, K = T * k, case["K"]
        q, p = quantised64(s["x"].double(), 8)
        codes = torch.zeros((R, K), dtype=torch.float64, device="cuda")
        S = torch.ones((R, K // 32), dtype=torch.float64, device="cuda")
        for j in range(k):
            took = s["slot_row"][:, j] >= 0
            codes[s["slot_row"][took, j].long()] = q[took]
            S[s["slot_row"][took, j].long()] = p[took]
        return dict(codes=codes, scales=placed(s["scales"], S, K))
    f64 = torch.float64

    def joined64(y):
        b = torch.zeros((T, y.shape[1]), dtype=f64, device="cuda")
        for j in range(k):
            took = s["slot_row"][:, j] >= 0
            b[took] += s["gates"][took, j, None].double() * y[s["slot_row"][took, j].long()]
        if s.get("w_post") is not None:
            b = b / torch.sqrt((b * b).mean(1, keepdim=True) + EPS) * s["w_post"].double()
        h = s["resid"].double() + 0.5 * b
        return dict(h=h, n=h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * s["w_pre"].double())

    if op == "combine":
        return joined64(s["y"].double())
    E, K, R = case["E"], case["K"], T * k
    rows = int(counts(case).sum())
    if rows * K * (case.get("N") or 3 * case["F"]) > 4e12:
        return None
    if op == "gemm":
        A = values4(s["A"], s["SA"], f64)
        return one_by_one(lambda e, a, b: A[a:b] @ values4(s["B"][e], s["SB"][e], f64).T, torch.zeros((R, case["N"]), dtype=f64, device="cuda"), E)
    F = case["F"]

    def hidden(A, weights):
        def f(e, a, b):
            g, u = A[a:b] @ weights(e, 0).T, A[a:b] @ weights(e, 1).T
            return g * torch.sigmoid(g) * u
        return one_by_one(f, torch.zeros((R, F), dtype=f64, device="cuda"), E)

    if op == "swiglu":
        h = hidden(values8(s["A"], s["SA"], f64), lambda e, i: values8(s["B"][e, i], s["SB"][e, i], f64))
        q, p = quantised64(h, 8)
        return dict(codes=q, scales=placed(s["scales"], p, F))
    q, p = quantised64(s["x"].double(), 4)
    x = (q.view(T, -1, 32) * p[..., None]).view(T, K)
    A = torch.zeros((R, K), dtype=f64, device="cuda")
    for j in range(k):
        took = s["slot_row"][:, j] >= 0
        A[s["slot_row"][took, j].long()] = x[took]
    h = hidden(A, lambda e, i: values4(s["B1"][e, i], s["S1"][e, i], f64))
    q, p = quantised64(h, 4)
    H = (q.view(R, -1, 32) * p[..., None]).view(R, F)
    y = one_by_one(lambda e, a, b: H[a:b] @ values4(s["B2"][e], s["S2"][e], f64).T, torch.zeros((R, K), dtype=f64, device="cuda"), E)
    return joined64(y)
