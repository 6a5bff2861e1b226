"""Cases that time the operators of a dense feed-forward layer in training and serving.

Five operators, each with a plain form in elementary torch operations (32-bit
arithmetic, one rounding at the end) and the library's own calls:

  linear      z = alpha A . B^T + bias on block-scaled operands; d = act(z) +
              res_scale R, as bf16 or quantised for the next product; z itself
              in 8 bits where the backward pass needs it
  checkpoint  bf16 rows -> MXFP8 in two orientations, blocks along the rows and
              blocks along the columns (the operand of a weight gradient), and
              the column sums (a bias gradient)
  backward    from dh and the 8-bit z: dz = dh act'(z) in both orientations, the
              bias gradient, and h = act(z) again, blocks along the columns
  norm        layer norm of bf16 rows, with the rows' statistics
  norm_grad   its gradients: dx (plus the residual stream's), dw, db

What is held in 8 bits is returned as the float8 values it stands for (codes
as E4M3 or E5M2, scales as E8M0).
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")     # in the order of the library's codes
FORMATS = {"e4m3": (0, torch.float8_e4m3fn, 8, 448.0, 3, -6), "e5m2": (1, torch.float8_e5m2, 15, 57344.0, 2, -14)}
EPS = 1e-5


def listed():
    return [
        # One token of a serving loop through a gated-less up projection: the weights' bytes rule.
        dict(name="linear decode", op="linear", form="mxfp4", M=1, N=8192, K=8192, bias="bf16", act="silu", resid=False, out="d", keep=False),
        # A ragged batch's down projection on byte operands, added to the residual stream.
        dict(name="linear ragged batch", op="linear", form="mxfp8", M=333, N=4010, K=4096, bias="fp32", act="none", resid=True, out="d", keep=False),
        # A prefill's up projection on packed operands.
        dict(name="linear prefill", op="linear", form="mxfp4", M=8192, N=8192, K=8192, bias="bf16", act="gelu_tanh", resid=False, out="d", keep=False),
        # A training step's up projection: the hidden rows quantised for the next product, z kept in 8 bits.
        dict(name="linear training", op="linear", form="mxfp8", M=8192, N=8192, K=4096, bias="fp32", act="gelu", resid=False, out="h", keep=True),
        # A small batch's rows, kept for the weight gradient.
        dict(name="checkpoint batch", op="checkpoint", rows=77, cols=1024, fmt="e4m3", sums=False),
        # A training step's output gradient, both orientations and the bias gradient.
        dict(name="checkpoint training", op="checkpoint", rows=16384, cols=8192, fmt="e5m2", sums=True),
        # The activation's backward pass of a small batch.
        dict(name="backward batch", op="backward", rows=500, cols=2048, act="silu", fmt="e4m3", fmt_z="e4m3"),
        # And of a training step: 8192 tokens, the hidden width of a 4096-wide layer.
        dict(name="backward training", op="backward", rows=8192, cols=16384, act="gelu", fmt="e5m2", fmt_z="e4m3"),
        # One token's norm: pure latency.
        dict(name="norm decode", op="norm", T=1, N=8192, param="bf16"),
        # A training step's rows.
        dict(name="norm training", op="norm", T=16384, N=8192, param="fp32"),
        # A small batch with rows of an odd width.
        dict(name="norm gradient batch", op="norm_grad", T=300, N=1001, param="fp32", resid=False),
        # A training step's gradients, the residual stream's added.
        dict(name="norm gradient training", op="norm_grad", T=16384, N=8192, param="bf16", resid=True),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["linear", "linear", "linear", "checkpoint", "backward", "norm", "norm_grad"])
    act = rng.choice(ACTS)
    fmt = rng.choice(["e4m3", "e5m2"])
    if op == "linear":
        form = rng.choice(["mxfp4", "mxfp8"])
        out = rng.choice(["d", "h"]) if form == "mxfp8" else "d"
        n = log(64, 8192)
        return dict(op=op, form=form, M=log(1, 8192), N=32 * max(1, n // 32) if out == "h" else n, K=32 * log(1, 256), act=act, out=out,
                    bias=rng.choice(["none", "bf16", "fp32"]), resid=rng.random() < 0.5, keep=rng.random() < 0.5)
    if op == "checkpoint":
        return dict(op=op, rows=log(1, 16384), cols=log(32, 8192), fmt=fmt, sums=rng.random() < 0.5)
    if op == "backward":
        return dict(op=op, rows=log(1, 8192), cols=log(32, 16384), act=act, fmt=fmt, fmt_z=rng.choice(["e4m3", "e5m2"]))
    if op == "norm":
        return dict(op=op, T=log(1, 16384), N=log(16, 8192), param=rng.choice(["bf16", "fp32"]))
    return dict(op=op, T=log(1, 16384), N=log(16, 8192), param=rng.choice(["bf16", "fp32"]), resid=rng.random() < 0.5)


def up32(n):
    return -(-n // 32) * 32


# ------------------------------------------------------------------ the inputs --


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = "cuda"
    bf16, u8 = torch.bfloat16, torch.uint8

    def normal(*shape, scale=1.0, dtype=bf16):
        return torch.randn(shape, device=dev, generator=g).mul_(scale).to(dtype)

    def empty(*shape, dtype=u8):
        return torch.empty(shape, dtype=dtype, device=dev)

    def operand4(rows, K):
        """Packed E2M1 rows of normal values, a scale for each 32."""
        limits = torch.tensor([(a + b) / 2 for a, b in zip(E2M1, E2M1[1:])], device=dev)
        x = torch.randn((rows, K // 2, 2), device=dev, generator=g).mul_(2.5)
        c = torch.bucketize(x.abs(), limits).to(u8) | (x < 0).to(u8) << 3
        return c[..., 0] | c[..., 1] << 4, torch.randint(126, 129, (rows, K // 32), dtype=u8, device=dev, generator=g)

    def operand8(rows, K):
        x = torch.randn((rows, K), device=dev, generator=g).mul_(100).clamp_(-448, 448)
        return x.to(torch.float8_e4m3fn).view(u8), torch.randint(120, 123, (rows, K // 32), dtype=u8, device=dev, generator=g)

    def parameter(n, kind, mean=0.0, scale=0.2):
        return None if kind == "none" else (normal(n, scale=scale, dtype=torch.float32) + mean).to(bf16 if kind == "bf16" else torch.float32)

    op = case["op"]
    s = {"case": case}
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        make = operand4 if case["form"] == "mxfp4" else operand8
        s["A"], s["SA"] = make(M, K)
        s["B"], s["SB"] = make(N, K)
        spread = 6.6 if case["form"] == "mxfp4" else 100.0 ** 2 / 2 ** 11     # of a product of two elements, scales included
        s["alpha"] = 1.5 / (spread * math.sqrt(K))
        s["bias"] = parameter(N, case["bias"])
        s["R"] = normal(M, N) if case["resid"] else None
        s["D"] = empty(M, N, dtype=bf16) if case["out"] == "d" else None
        s["H"], s["SH"] = (empty(M, N), empty(M, N // 32)) if case["out"] == "h" else (None, None)
        s["Z"], s["SZ"] = (empty(M, up32(N)), empty(M, up32(N) // 32)) if case["keep"] else (None, None)
        s["workspace"] = empty(64 << 20)
    elif op in ("checkpoint", "backward"):
        rows, cols = case["rows"], case["cols"]
        pad = up32(cols) - cols

        def wide(scale):
            """Rows as gradients and activations are: a few channels and tokens much larger."""
            x = torch.randn((rows, cols), device=dev, generator=g).mul_(scale)
            x *= 1 + 7 * (torch.rand((1, cols), device=dev, generator=g) < 0.01)
            x *= torch.exp(torch.randn((rows, 1), device=dev, generator=g))
            return torch.nn.functional.pad(x.to(bf16), (0, pad))

        s["x"] = wide(1.0 if op == "checkpoint" else 1e-3)[:, :cols]
        s["Q"], s["S"] = empty(rows, up32(cols)), empty(rows, up32(cols) // 32)
        s["QT"], s["ST"] = empty(cols, up32(rows)), empty(cols, up32(rows) // 32)
        s["sums"] = empty(cols, dtype=torch.float32) if op == "backward" or case["sums"] else None
        if op == "backward":
            code, kind, emax, most, _, _ = FORMATS[case["fmt_z"]]
            z = torch.randn((rows, up32(cols)), device=dev, generator=g).mul_(1.7)
            z[:, cols:] = 0
            e = torch.frexp(z.unflatten(1, (-1, 32)).abs().amax(-1))[1] - 1 - emax
            e = torch.where(z.unflatten(1, (-1, 32)).abs().amax(-1) == 0, 0, e)
            s["SZ"] = (e + 127).to(u8)
            s["Z"] = (z.unflatten(1, (-1, 32)) * torch.exp2(-e.float())[..., None]).flatten(1).clamp(-most, most).to(kind).view(u8)
            s["HT"], s["SHT"] = empty(cols, up32(rows)), empty(cols, up32(rows) // 32)
        s["workspace"] = empty(64 << 20)
    else:
        T, N = case["T"], case["N"]
        x = torch.randn((T, N), device=dev, generator=g) + 0.3 * torch.randn((T, 1), device=dev, generator=g)
        x *= 1 + 7 * (torch.rand((1, N), device=dev, generator=g) < 0.01)
        s["x"] = x.to(bf16)
        s["w"] = parameter(N, case["param"], mean=1.0)
        if op == "norm":
            s["b"] = parameter(N, case["param"])
            s["y"], s["mean"], s["rstd"] = empty(T, N, dtype=bf16), empty(T, dtype=torch.float32), empty(T, dtype=torch.float32)
        else:
            wide = s["x"].double()
            s["mean"] = wide.mean(1).float()
            s["rstd"] = torch.rsqrt(wide.var(1, unbiased=False) + EPS).float()
            s["dy"] = normal(T, N, scale=1e-2)
            s["dres"] = normal(T, N, scale=1e-2) if case["resid"] else None
            s["dx"], s["dw"], s["db"] = empty(T, N, dtype=bf16), empty(N, dtype=torch.float32), empty(N, dtype=torch.float32)
            s["workspace"] = empty(64 << 20)
    return s


# ------------------------------------------------------------------ the plain forms --


def two_to(e):
    """2^e for whole e from -126 to 127, exactly, in 32 bits."""
    return ((e.int() + 127) << 23).view(torch.float32)


def scaled(v, s):
    """Values [.., K] times their blocks' scales [.., K / 32] (E8M0 codes 1 to 254)."""
    return (v.unflatten(-1, (-1, 32)) * two_to(s.int() - 127)[..., None]).flatten(-2)


def values4(q, s):
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=q.device)
    return scaled(torch.stack((lut[(q & 15).int()], lut[(q >> 4).int()]), -1).flatten(-2), s)


def values8(q, s, fmt="e4m3"):
    return scaled(q.view(FORMATS[fmt][1]).float(), s)


def quantised(x, fmt):
    """Rows [R, K] -> codes [R, K up to whole blocks] and scales: 2^(floor(log2 amax) - emax), 1 for zeros."""
    _, kind, emax, most, _, _ = FORMATS[fmt]
    x = torch.nn.functional.pad(x, (0, up32(x.shape[1]) - x.shape[1])).unflatten(1, (-1, 32))
    amax = x.abs().amax(-1)
    e = torch.where(amax == 0, 0, (torch.frexp(amax)[1] - 1 - emax).clamp(-127, 127))
    q = (x * two_to(-e)[..., None]).clamp(-most, most).to(kind)
    return q.flatten(1), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def act(z, kind):
    if kind == "relu":
        return z * (z > 0)
    if kind == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    if kind == "gelu_tanh":                                  # (1 + tanh(u)) / 2 = 1 / (1 + exp(-2 u)), without cancellation
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if kind == "silu":
        return z / (1 + torch.exp(-z))
    return z


def act_slope(z, kind):
    if kind == "relu":
        return (z > 0).to(z.dtype)
    if kind == "gelu":
        return 0.5 * torch.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        g = 1 / (1 + torch.exp(-c * (z + 0.044715 * z * z * z)))
        return g * (1 + z * (1 - g) * c * (1 + 3 * 0.044715 * z * z))
    if kind == "silu":
        g = 1 / (1 + torch.exp(-z))
        return g * (1 + z * (1 - g))
    return torch.ones_like(z)


def plain(s):
    case = s["case"]
    op = case["op"]
    if op == "linear":
        values = values4 if case["form"] == "mxfp4" else values8
        z = s["alpha"] * torch.matmul(values(s["A"], s["SA"]), values(s["B"], s["SB"]).t())
        if s["bias"] is not None:
            z = z + s["bias"].float()
        d = act(z, case["act"])
        if s["R"] is not None:
            d = d + 0.5 * s["R"].float()
        out = dict(d=d.to(torch.bfloat16)) if case["out"] == "d" else dict(zip(("h", "sh"), quantised(d, "e4m3")))
        if case["keep"]:
            out["z"], out["sz"] = quantised(z, "e4m3")
        return out
    if op == "checkpoint":
        x = s["x"].float()
        out = dict(zip(("q", "s", "qt", "st"), (*quantised(x, case["fmt"]), *quantised(x.t(), case["fmt"]))))
        if case["sums"]:
            out["sums"] = x.sum(0)
        return out
    if op == "backward":
        z = values8(s["Z"], s["SZ"], case["fmt_z"])[:, :case["cols"]]
        dz = s["x"].float() * act_slope(z, case["act"])
        out = dict(zip(("q", "s", "qt", "st"), (*quantised(dz, case["fmt"]), *quantised(dz.t(), case["fmt"]))))
        out["ht"], out["sht"] = quantised(act(z, case["act"]).t(), "e4m3")
        return dict(out, sums=dz.sum(0))
    x, w = s["x"].float(), s["w"].float()
    if op == "norm":
        mean = x.mean(1, keepdim=True)
        rstd = torch.rsqrt((x - mean).square().mean(1, keepdim=True) + EPS)
        y = (x - mean) * rstd * w + s["b"].float()
        return dict(y=y.to(torch.bfloat16), mean=mean[:, 0], rstd=rstd[:, 0])
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xhat = (x - s["mean"][:, None]) * rstd
    v = dy * w
    dx = rstd * (v - v.mean(1, keepdim=True) - xhat * (v * xhat).mean(1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return dict(dx=dx.to(torch.bfloat16), dw=(dy * xhat).sum(0), db=dy.sum(0))


# ------------------------------------------------------------------ the library's calls --


def library(s):
    import block_scaled_mxfp4_gb300 as mx

    def ld(t):
        return 0 if t is None else t.stride(0) if t.shape[0] > 1 else t.shape[1]

    def codes(t, fmt):
        return t.view(FORMATS[fmt][1])

    def scales(t):
        return t.view(torch.float8_e8m0fnu)

    case, ws = s["case"], s.get("workspace")
    op = case["op"]
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        kind = mx.MXFP4_PARAM_FP32 if case["bias"] == "fp32" else mx.MXFP4_PARAM_BF16
        rest = (s["alpha"], s["bias"], kind, ACTS.index(case["act"]), s["R"], N, 0.5, M, N, K, 0, 0, ws, ws.numel())
        if case["form"] == "mxfp4":
            mx.mxfp4_gemm_act(s["D"], N, None, 0, None, 0, s["Z"], up32(N), s["SZ"], up32(N) // 32, s["A"], K, s["B"], K,
                              s["SA"], K // 32, s["SB"], K // 32, mx.MXFP8_E4M3, *rest)
        else:
            mx.mxfp8_gemm_act(s["D"], N, s["H"], N, s["SH"], N // 32, s["Z"], up32(N), s["SZ"], up32(N) // 32, s["A"], K, s["B"], K,
                              s["SA"], K // 32, s["SB"], K // 32, mx.MXFP8_E4M3, mx.MXFP8_E4M3, mx.MXFP8_E4M3, mx.MXFP8_E4M3, *rest)
        out = dict(d=s["D"]) if case["out"] == "d" else dict(h=codes(s["H"], "e4m3"), sh=scales(s["SH"]))
        if case["keep"]:
            out["z"], out["sz"] = codes(s["Z"], "e4m3"), scales(s["SZ"])
        return out
    if op in ("checkpoint", "backward"):
        rows, cols, fmt = case["rows"], case["cols"], case["fmt"]
        both = (s["Q"], up32(cols), s["S"], up32(cols) // 32, s["QT"], up32(rows), s["ST"], up32(rows) // 32)
        out = dict(q=codes(s["Q"], fmt), s=scales(s["S"]), qt=codes(s["QT"], fmt), st=scales(s["ST"]))
        if op == "checkpoint":
            mx.mxfp8_checkpoint(*both, s["sums"], s["x"], up32(cols), rows, cols, FORMATS[fmt][0], ws, ws.numel())
        else:
            mx.mxfp8_act_backward(None, 0, *both, s["HT"], up32(rows), s["SHT"], up32(rows) // 32, s["sums"], s["x"], up32(cols), s["Z"],
                                  up32(cols), s["SZ"], up32(cols) // 32, FORMATS[case["fmt_z"]][0], ACTS.index(case["act"]), rows, cols,
                                  FORMATS[fmt][0], mx.MXFP8_E4M3, ws, ws.numel())
            out["ht"], out["sht"] = codes(s["HT"], "e4m3"), scales(s["SHT"])
        if s["sums"] is not None:
            out["sums"] = s["sums"]
        return out
    T, N = case["T"], case["N"]
    kind = mx.MXFP4_PARAM_FP32 if case["param"] == "fp32" else mx.MXFP4_PARAM_BF16
    if op == "norm":
        mx.mxfp4_layer_norm(s["y"], N, s["mean"], s["rstd"], s["x"], N, s["w"], s["b"], kind, EPS, T, N)
        return dict(y=s["y"], mean=s["mean"], rstd=s["rstd"])
    mx.mxfp4_layer_norm_backward(s["dx"], N, s["dw"], s["db"], s["dy"], N, s["x"], N, s["mean"], s["rstd"], s["w"], kind, s["dres"],
                                 ld(s["dres"]), T, N, ws, ws.numel())
    return dict(dx=s["dx"], dw=s["dw"], db=s["db"])


def run(state):
    return library(state) if own else plain(state)


def work(case):
    op = case["op"]
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        element = 0.5 if case["form"] == "mxfp4" else 1.0
        read = (M + N) * K * (element + 1 / 32) + N * dict(none=0, bf16=2, fp32=4)[case["bias"]] + 2 * M * N * case["resid"]
        write = M * N * (2 if case["out"] == "d" else 1 + 1 / 32) + M * up32(N) * (1 + 1 / 32) * case["keep"]
        return {"bytes": read + write, "flops": 2 * M * N * K}
    if op in ("checkpoint", "backward"):
        rows, cols = case["rows"], case["cols"]
        by_row, by_col, q = rows * up32(cols), cols * up32(rows), 1 + 1 / 32
        if op == "checkpoint":
            return {"bytes": 2 * rows * cols + q * (by_row + by_col) + 4 * cols * case["sums"], "flops": 8 * rows * cols}
        return {"bytes": 2 * rows * cols + q * (2 * by_row + 2 * by_col) + 4 * cols, "flops": 32 * rows * cols}
    T, N = case["T"], case["N"]
    parameter = N * (2 if case["param"] == "bf16" else 4)
    if op == "norm":
        return {"bytes": 4 * T * N + 2 * parameter + 8 * T, "flops": 8 * T * N}
    return {"bytes": (8 if case["resid"] else 6) * T * N + parameter + 8 * N + 8 * T, "flops": 16 * T * N}


# ------------------------------------------------------------------ the definitions, in 64 bits --


def power(e):
    """2^e for whole e, in 64 bits, from its bits (a pow() may be a unit off)."""
    return (e.long() + 1023 << 52).view(torch.float64)


def decoded(q, s, fmt, K):
    """Codes as bytes [R, >= K] and E8M0 bytes -> float64 [R, K], from the fields of the code."""
    _, _, _, _, mbits, emin = FORMATS[fmt]
    q = q.long()
    e = (q & 127) >> mbits
    m = (q & ((1 << mbits) - 1)).double()
    v = torch.where(e == 0, m, m + (1 << mbits)) * power(torch.where(e == 0, 1, e) + emin - 1 - mbits)
    v = torch.where(q >= 128, -v, v)
    return (v * power(s.long() - 127).repeat_interleave(32, 1))[:, :K]


def decoded4(q, s):
    c = torch.stack((q & 15, q >> 4), -1).flatten(1).long()
    e, m = (c >> 1) & 3, (c & 1).double()
    v = torch.where(e == 0, m / 2, (1 + m / 2) * power(e - 1))
    return torch.where(c >= 8, -v, v) * power(s.long() - 127).repeat_interleave(32, 1)


def rounded(x, fmt):
    """float64 rows -> the nearest codes' values before scaling, and the scales, by the definition."""
    _, kind, emax, most, mbits, emin = FORMATS[fmt]
    R, K = x.shape
    block = x.new_zeros((R, up32(K)))
    block[:, :K] = x
    block = block.reshape(R, -1, 32)

    def binade(v):
        return (v.abs().view(torch.int64) >> 52) - 1023

    amax = block.abs().max(2).values
    e = torch.where(amax > 0, (binade(amax) - emax).clamp(-127, 127), 0)
    y = block * power(-e)[..., None]
    step = power(binade(y).clamp(min=emin) - mbits)
    y = (torch.round(y / step) * step).clamp(-most, most)
    return y.reshape(R, -1).to(kind), power(e).to(torch.float8_e8m0fnu)


def act64(z, kind):
    """act(z) and its slope."""
    if kind == "relu":
        return torch.clamp(z, min=0), torch.where(z > 0, 1.0, 0.0).double()
    if kind == "gelu":
        phi = torch.special.ndtr(z)
        return z * phi, phi + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        u = math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3)      # (1 + tanh(u / 2)) / 2 = sigmoid(u)
        g = torch.sigmoid(u)
        return z * g, g + z * g * torch.sigmoid(-u) * math.sqrt(8 / math.pi) * (1 + 0.134145 * z * z)
    if kind == "silu":
        g = torch.sigmoid(z)
        return z * g, g + z * g * torch.sigmoid(-z)
    return z, torch.ones_like(z)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        if case["form"] == "mxfp4":
            A, B = decoded4(s["A"], s["SA"]), decoded4(s["B"], s["SB"])
        else:
            A, B = decoded(s["A"], s["SA"], "e4m3", case["K"]), decoded(s["B"], s["SB"], "e4m3", case["K"])
        z = (A @ B.T).mul_(s["alpha"])
        if s["bias"] is not None:
            z += s["bias"].double()
        d = act64(z, case["act"])[0]
        if s["R"] is not None:
            d = d + s["R"].double() / 2
        out = {}
        if case["out"] == "d":
            out["d"] = d
        else:
            out["h"], out["sh"] = rounded(d, "e4m3")
        if case["keep"]:
            out["z"], out["sz"] = rounded(z, "e4m3")
        return out
    if op == "checkpoint":
        x = s["x"].double()
        (q, a), (qt, b) = rounded(x, case["fmt"]), rounded(x.T.contiguous(), case["fmt"])
        return dict(q=q, s=a, qt=qt, st=b, sums=x.sum(0) if case["sums"] else None)
    if op == "backward":
        z = decoded(s["Z"], s["SZ"], case["fmt_z"], case["cols"])
        h, slope = act64(z, case["act"])
        dz = s["x"].double() * slope
        (q, a), (qt, b), (ht, c) = rounded(dz, case["fmt"]), rounded(dz.T.contiguous(), case["fmt"]), rounded(h.T.contiguous(), "e4m3")
        return dict(q=q, s=a, qt=qt, st=b, ht=ht, sht=c, sums=dz.sum(0))
    x, w = s["x"].double(), s["w"].double()
    if op == "norm":
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = (var + EPS) ** -0.5
        return dict(y=(x - mean[:, None]) * (rstd[:, None] * w) + s["b"].double(), mean=mean, rstd=rstd)
    rstd = s["rstd"].double()
    xhat = (x - s["mean"].double()[:, None]) * rstd[:, None]
    dy = s["dy"].double()
    v = dy * w
    along = (v * xhat).sum(1) / case["N"]
    dx = (v - (v.sum(1) / case["N"])[:, None] - xhat * along[:, None]) * rstd[:, None]
    if s["dres"] is not None:
        dx = dx + s["dres"].double()
    return dict(dx=dx, dw=(dy * xhat).sum(0), db=dy.sum(0))
