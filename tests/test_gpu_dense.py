"""The dense layer's operators on the GPU through the C ABI against plain
64-bit forms (tests/dense_ref.py has the bounds and where they come from).

A product's accumulation is the dense GEMMs': within 2^-20 sum |a b|; with the
activations' largest slope, 1.13, that goes through them.
"""
import numpy as np
import pytest

import block_scaled_mxfp4_gb300 as mx
import dense_ref as dr
import expert_ref as ref
from block_scaled_mxfp4_gb300 import inputs
from dense_ref import EPS24, up32

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

FMT = {"e4m3": mx.MXFP8_E4M3, "e5m2": mx.MXFP8_E5M2}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from block_scaled_mxfp4_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    mx.mxfp4_device_status(reset=True)
    yield
    assert mx.mxfp4_device_status() == 0, "a bounded wait timed out during the tests"


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    torch.cuda.synchronize()
    return None if t is None else t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def bf16(x, ld=None, shift=0):
    """float64 rows -> (bf16 rows on the GPU, ld apart, `shift` elements off the allocation), their values."""
    x = torch.from_numpy(np.asarray(x, np.float64)).to(torch.bfloat16)
    rows, cols = x.shape
    ld = ld or cols
    flat = torch.full((rows * ld + shift + 16,), 777.0, dtype=torch.bfloat16, device="cuda")
    t = torch.as_strided(flat, (rows, cols), (ld, 1), shift)
    t.copy_(x)
    return t, x.double().numpy()


def u8(rows, ld, fill=0xEE):
    return torch.full((rows, ld), fill, dtype=torch.uint8, device="cuda")


def workspace(n):
    return torch.full((max(n, 256),), 0xAB, dtype=torch.uint8, device="cuda")


def param(x, kind):
    if x is None:
        return None, None
    t = torch.from_numpy(np.asarray(x, np.float64)).to(torch.bfloat16 if kind == "bf16" else torch.float32)
    return t.cuda(), t.double().numpy()


KIND = {"bf16": mx.MXFP4_PARAM_BF16, "fp32": mx.MXFP4_PARAM_FP32}

# ----------------------------------------------------------------- products --


class Product:
    def __init__(self, form, M, N, K, seed=0):
        self.form, self.M, self.N, self.K = form, M, N, K
        if form == "mxfp4":
            p = inputs.make_problem("act", M, N, K, seed, "normal", 1.0, 0.0, None)
            fa = fb = "e2m1"
        else:
            fa, fb = ("e4m3", "e5m2") if form == "mixed" else ("e4m3", "e4m3")
            p = inputs.make_problem8("act", M, N, K, seed, fa, fb, "normal", 1.0, 0.0, None)
        self.A, self.B = ref.values(p.A, p.SA, fa), ref.values(p.B, p.SB, fb)
        self.fmts = [FMT.get(f) for f in (fa, fb)]
        self.dA, self.dB, self.dSA, self.dSB = dev(p.A), dev(p.B), dev(p.SA), dev(p.SB)
        self.acc = self.A @ self.B.T
        self.mag = np.abs(self.A) @ np.abs(self.B).T
        self.alpha = float(np.float32(1.5 / max(1e-30, np.sqrt((self.acc ** 2).mean()))))

    def run(self, act="none", bias=None, bias_kind="bf16", R=None, res_scale=1.0, d=True, h=None, z=None, split_k=0, flags=0,
            ldd=None, ldh=None, ldz=None, stream=None, alpha=None, D=None, extra=3):
        M, N, K = self.M, self.N, self.K
        packed = self.form == "mxfp4"
        if d and D is None:
            D = torch.full((M, ldd or N), 777.0, dtype=torch.bfloat16, device="cuda")
        ldh = ldh or up32(N)
        H, SH = (u8(M, ldh // 2 if packed else ldh), u8(M, up32(N) // 32 + extra, 0xDD)) if h else (None, None)
        ldz = ldz or up32(N)
        Z, SZ = (u8(M, ldz), u8(M, up32(N) // 32 + extra, 0xDD)) if z else (None, None)
        size = mx.mxfp4_gemm_workspace_size if packed else mx.mxfp8_gemm_workspace_size
        need = size(M, N, K, split_k)
        ws = workspace(need)
        front = (D if d else None, D.stride(0) if d else 0, H, ldh, SH, up32(N) // 32 + extra, Z, ldz, SZ, up32(N) // 32 + extra,
                 self.dA, K, self.dB, K, self.dSA, K // 32, self.dSB, K // 32)
        back = (self.alpha if alpha is None else alpha, bias, KIND[bias_kind], dr.ACTS.index(act), R, R.stride(0) if R is not None else 0,
                res_scale, M, N, K, split_k, flags, ws, need)
        if packed:
            mx.mxfp4_gemm_act(*front, FMT[z or "e4m3"], *back, stream=stream)
        else:
            mx.mxfp8_gemm_act(*front, *self.fmts, FMT[h or "e4m3"], FMT[z or "e4m3"], *back, stream=stream)
        return D, H, SH, Z, SZ

    def check(self, act="none", bias=False, bias_kind="bf16", resid=False, h=None, z=None, d=True, res_scale=0.5, alpha=None, **kw):
        rng = np.random.default_rng(self.M + self.N)
        db, b = param(rng.normal(size=self.N) * 0.3, bias_kind) if bias else (None, 0.0)
        dR, R = bf16(rng.normal(size=(self.M, self.N)), ld=self.N + 5 if resid == "apart" else None) if resid else (None, 0.0)
        out = self.run(act, db, bias_kind, dR, res_scale, d, h, z, alpha=alpha, **kw)
        alpha = self.alpha if alpha is None else alpha
        Z = alpha * self.acc + b
        ez = abs(alpha) * 2.0 ** -20 * self.mag + 2 * EPS24 * np.abs(Z)
        H, _, eh, _ = dr.act(Z, act)
        V = H + res_scale * R
        ev = 1.13 * ez + eh + 2 * EPS24 * (np.abs(V) + np.abs(H))
        D, Hq, SH, Zq, SZ = map(host, out)
        if d:
            dr.check_bf16(D[:, :self.N], V, ev, "D")
            assert (D[:, self.N:] == 776.0).all()
        if h:
            dr.check_codes(Hq, SH, V, ev, "e2m1" if self.form == "mxfp4" else h, "H")
        if z:
            dr.check_codes(Zq, SZ, Z, ez, z, "Z")
        return out


# The kernels and plans: CTA pairs; one tile of 256, 128 and 64 columns; swapped
# operands; splits reduced in a cluster and in the workspace; tiles cut at M, N and K.
PLANS = [("mxfp4", 2560, 2304, 512, 0), ("mxfp4", 2309, 2500, 288, 0), ("mxfp8", 700, 1100, 384, 0), ("mxfp8", 300, 96, 160, 0),
         ("mxfp4", 200, 40, 320, 0), ("mxfp4", 1, 256, 512, 0), ("mxfp8", 5, 1000, 2048, 0), ("mxfp8", 64, 333, 4096, 0),
         ("mxfp4", 33, 160, 8192, 0), ("mxfp4", 300, 500, 4096, 4), ("mxfp8", 130, 290, 2048, 5), ("mxfp8", 257, 129, 1024, 8),
         ("mxfp4", 7, 97, 8192, 3), ("mxfp8", 40, 64, 2048, 7), ("mxfp8", 140, 200, 4096, 11), ("mxfp4", 9, 200, 8192, 16),
         ("mixed", 1, 1, 32, 0), ("mixed", 65, 3, 64, 0), ("mixed", 3, 2, 32, 0), ("mxfp8", 128, 256, 128, 0),
         ("mxfp8", 2560, 2304, 512, 0), ("mixed", 2309, 2501, 416, 0), ("mxfp8", 1000, 4999, 64, 0)]


@pytest.fixture(scope="module")
def products():
    made = {}

    def get(form, M, N, K):
        if (form, M, N, K) not in made:
            made[form, M, N, K] = Product(form, M, N, K, M + N)
        return made[form, M, N, K]
    return get


@pytest.mark.parametrize("act", dr.ACTS)
@pytest.mark.parametrize("form,M,N,K,split", PLANS)
def test_product(products, form, M, N, K, split, act):
    p = products(form, M, N, K)
    p.check(act, bias=True, bias_kind="fp32" if act in ("gelu", "none") else "bf16", resid=act in ("none", "silu"), split_k=split)


@pytest.mark.parametrize("form,M,N,K,split", PLANS)
@pytest.mark.parametrize("z", ["e4m3", "e5m2"])
def test_product_keeps_z(products, form, M, N, K, split, z):
    p = products(form, M, N, K)
    p.check("gelu" if z == "e4m3" else "silu", bias=z == "e4m3", z=z, split_k=split, ldz=up32(N) + (16 if z == "e5m2" else 0))
    p.check("relu", z=z, d=False, split_k=split)


@pytest.mark.parametrize("form,M,N,K,split", [p for p in PLANS if p[2] % 32 == 0])
@pytest.mark.parametrize("h", ["e4m3", "e5m2"])
def test_product_quantises_d(products, form, M, N, K, split, h):
    p = products(form, M, N, K)
    p.check("gelu_tanh", bias=True, resid="apart", h=h, z=h, split_k=split, ldh=N + 32)
    p.check("none", h=h, d=False, split_k=split)


def test_product_forms_of_one_call_agree(products):
    """Each output alone has the bits that it has beside the others."""
    p = products("mxfp8", 700, 1100, 384)
    D, _, _, Z, SZ = p.check("silu", z="e4m3")
    D1 = p.check("silu")[0]
    Z1 = p.check("silu", z="e4m3", d=False)[3]
    assert torch.equal(D, D1) and torch.equal(Z, Z1)


@pytest.mark.parametrize("form,M,N,K,split", [PLANS[i] for i in (0, 2, 5, 7, 8, 9, 11, 14, 15, 20, 21)])
def test_product_without_epilogue_is_the_gemm(products, form, M, N, K, split):
    p = products(form, M, N, K)
    got = p.run(split_k=split)[0]
    want = torch.empty_like(got)
    size = mx.mxfp4_gemm_workspace_size if form == "mxfp4" else mx.mxfp8_gemm_workspace_size
    ws = workspace(size(M, N, K, split))
    args = (want, N, None, 0, p.dA, K, p.dB, K, p.dSA, K // 32, p.dSB, K // 32)
    if form == "mxfp4":
        mx.mxfp4_gemm(*args, p.alpha, 0.0, M, N, K, split, ws, ws.numel())
    else:
        mx.mxfp8_gemm(*args, *p.fmts, p.alpha, 0.0, M, N, K, split, ws, ws.numel())
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("form,M,N,K,split", [PLANS[i] for i in (0, 1, 2, 5, 7, 9, 10, 14, 15, 20, 21)])
def test_product_strides_and_residual_in_place(products, form, M, N, K, split):
    p = products(form, M, N, K)
    x = np.random.default_rng(1).normal(size=(M, N))
    for ld in (N + 8 - N % 8 + 8, N + 3):
        D, R = bf16(x, ld=ld)
        p.run("silu", R=D, D=D, res_scale=0.5, split_k=split)
        Z = p.alpha * p.acc
        ez = abs(p.alpha) * 2.0 ** -20 * p.mag + 2 * EPS24 * np.abs(Z)
        H, _, eh, _ = dr.act(Z, "silu")
        V = H + 0.5 * R
        dr.check_bf16(host(D), V, 1.13 * ez + eh + 2 * EPS24 * (np.abs(V) + np.abs(H)))
        around = torch.as_strided(D, (M, ld - N), (ld, 1), D.storage_offset() + N)
        assert (around[:-1] == 776.0).all()


@pytest.mark.parametrize("M,N,K", [(2560, 2304, 512), (1, 256, 512), (200, 40, 320), (300, 500, 4096)])
def test_product_extremes(products, M, N, K):
    """Large and tiny z of either sign, zeros, and blocks that are not finite."""
    p = products("mxfp4", M, N, K)
    for factor in (2.0 ** 6, 2.0 ** -60, 0.0):
        for act in dr.ACTS:
            p.check(act, alpha=float(np.float32(p.alpha * factor)), z="e4m3")
    keep = p.dSA.clone()
    p.dSA[M // 2] = 255                                      # a row of NaN
    D, H, SH, Z, SZ = map(host, p.run("gelu", z="e4m3"))
    assert np.isnan(D[M // 2]).all() and np.isnan(D).any(1).sum() == 1
    bad = SZ[:, :up32(N) // 32] == 255
    assert bad[M // 2].all() and bad.any(1).sum() == 1
    p.dSA = keep


def test_product_repeats_and_keeps_order(products):
    """Calls back to back, each reading what the one before wrote, and replays in a graph."""
    p = products("mxfp8", 64, 333, 4096)
    q = products("mxfp4", 2560, 2304, 512)
    want = [t.clone() for t in p.run("gelu", z="e4m3") if t is not None], [t.clone() for t in q.run("silu", h="e4m3") if t is not None]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for _ in range(3):
            got = [t for t in p.run("gelu", z="e4m3") if t is not None], [t for t in q.run("silu", h="e4m3") if t is not None]
    s.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    D, _ = bf16(np.zeros((p.M, p.N)))
    g = torch.cuda.CUDAGraph()
    ws = workspace(mx.mxfp8_gemm_workspace_size(p.M, p.N, p.K, 0))
    with torch.cuda.graph(g):
        for _ in range(2):
            mx.mxfp8_gemm_act(D, p.N, None, 0, None, 0, None, 0, None, 0, p.dA, p.K, p.dB, p.K, p.dSA, p.K // 32, p.dSB, p.K // 32,
                              0, 0, 0, 0, p.alpha, None, 0, mx.MXFP4_ACT_RELU, D, p.N, 1.0, p.M, p.N, p.K, 0, 0, ws, ws.numel())
    for n in range(1, 4):
        g.replay()
        torch.cuda.synchronize()
        relu = np.maximum(p.alpha * p.acc, 0)
        # 2 n additions, each rounded to half a bf16 step of a value of at most the last one's size.
        e = 2 * n * (p.alpha * 2.0 ** -20 * p.mag + 2.0 ** -9 * (2 * n + 1) * relu + 2.0 ** -60)
        assert (np.abs(host(D) - 2 * n * relu) <= e).all()


def test_product_static_weights(products):
    p = products("mxfp4", 33, 160, 8192)
    a = p.run("silu", z="e4m3")
    b = p.run("silu", z="e4m3", flags=mx.MXFP4_FLAG_B_STATIC)
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[3], b[3]) and torch.equal(a[4], b[4])


def test_product_offsets_past_32_bits():
    """Rows of D, R and Z more than 2^31 elements from the first."""
    M, N, K = 300, 64, 64
    p = Product("mxfp8", M, N, K, 4)
    ld = 1 << 23
    D = torch.empty((M, ld), dtype=torch.bfloat16, device="cuda")
    Z = torch.empty((M, ld), dtype=torch.uint8, device="cuda")
    SZ = torch.empty((M, 2), dtype=torch.uint8, device="cuda")
    D[:, :N] = 1.0
    mx.mxfp8_gemm_act(D, ld, None, 0, None, 0, Z, ld, SZ, 2, p.dA, K, p.dB, K, p.dSA, 2, p.dSB, 2, 0, 0, 0, 0, p.alpha, None, 0, 0, D, ld,
                      1.0, M, N, K, 0, 0, None, 0)
    V = p.alpha * p.acc
    e = p.alpha * 2.0 ** -20 * p.mag + 2 * EPS24 * (np.abs(V) + 1)
    dr.check_bf16(host(D[:, :N].contiguous()), V + 1, e)
    dr.check_codes(host(Z[:, :N].contiguous()), host(SZ), V, e, "e4m3")


# -------------------------------------------------------------- checkpoints --


def run_checkpoint(x, cols, fmt, row=True, col=True, sums=True, pad=0, stream=None, extra=2):
    rows = x.shape[0]
    Q, S = (u8(rows, up32(cols) + pad), u8(rows, up32(cols) // 32 + extra, 0xDD)) if row else (None, None)
    QT, ST = (u8(cols, up32(rows) + pad), u8(cols, up32(rows) // 32 + extra, 0xDD)) if col else (None, None)
    out = torch.full((cols,), float("nan"), device="cuda") if sums else None
    need = mx.mxfp8_checkpoint_workspace_size(rows, cols)
    ws = workspace(need)
    mx.mxfp8_checkpoint(Q, up32(cols) + pad, S, up32(cols) // 32 + extra, QT, up32(rows) + pad, ST, up32(rows) // 32 + extra, out, x,
                        x.stride(0), rows, cols, FMT[fmt], ws, need, stream=stream)
    return Q, S, QT, ST, out


def sum_bound(rows, v):
    """Chains of fp32 additions: a lane's rows, then lanes, warps and strips."""
    return (rows / 32 + 64) * EPS24 * np.abs(v).sum(0)


SIZES = [(1, 1), (1, 32), (2, 1000), (31, 33), (32, 64), (33, 31), (77, 1024), (129, 257), (500, 96), (1000, 1001), (4099, 72), (300, 2050)]


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_checkpoint(rows, cols, fmt):
    rng = np.random.default_rng(rows + cols)
    x = rng.normal(size=(rows, cols)) * np.exp(rng.normal(size=(rows, 1)) * 2) * np.exp(rng.normal(size=(1, cols)) * 2)
    x[rng.uniform(size=x.shape) < 0.05] = 0
    t, x = bf16(x, ld=-(-cols // 8) * 8 + 8)
    Q, S, QT, ST, sums = map(host, run_checkpoint(t, cols, fmt, pad=16))
    dr.check_codes(Q, S, x, 0, fmt, "rows")
    dr.check_codes(QT, ST, np.ascontiguousarray(x.T), 0, fmt, "columns")
    assert (np.abs(sums - x.sum(0)) <= sum_bound(rows, x)).all()


@pytest.mark.parametrize("rows,cols", [(77, 1024), (300, 2080)])
def test_checkpoint_outputs_alone(rows, cols):
    t, _ = bf16(np.random.default_rng(0).normal(size=(rows, cols)))
    whole = run_checkpoint(t, cols, "e4m3")
    for row, col, sums in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 0, 1)):
        for a, b in zip(whole, run_checkpoint(t, cols, "e4m3", row, col, sums)):
            assert b is None or torch.equal(a, b)
    # The row form is mxfp8_quantize's.
    Q, S = u8(rows, cols), u8(rows, cols // 32)
    mx.mxfp8_quantize(Q, cols, S, cols // 32, t, cols, rows, cols, mx.MXFP8_E4M3)
    assert torch.equal(Q, whole[0]) and torch.equal(S, whole[1][:, :cols // 32])
    # No workspace where nothing is summed.
    mx.mxfp8_checkpoint(Q, cols, S, cols // 32, None, 0, None, 0, None, t, cols, rows, cols, 0, None, 0)


def test_checkpoint_special_values():
    rows, cols = 96, 96
    x = np.random.default_rng(2).normal(size=(rows, cols))
    x[:, 5] = 0                                              # blocks of zeros
    x[7] = 0
    x[8] = -0.0
    x[9], x[:, 9] = 2.0 ** -130, 2.0 ** -126                  # subnormal numbers, the smallest scales
    x[10], x[:, 10] = 3.3e38, -3.3e38
    x[11] = 448.0 * np.where(np.arange(cols) % 2, 1, -1)
    x[12, :32] = np.tile([464, 465, 480, 511, -464, -465, 1, 2.0 ** -9], 4)
    for fmt in FMT:
        t, v = bf16(x)
        Q, S, QT, ST, _ = map(host, run_checkpoint(t, cols, fmt))
        dr.check_codes(Q, S, v, 0, fmt)
        dr.check_codes(QT, ST, np.ascontiguousarray(v.T), 0, fmt)
        assert (np.delete(Q[8], [9, 10]) == 0x80).all()     # (columns 9 and 10 hold values of their own)
    y = x.copy()
    y[3, 40], y[50, 70], y[70, 3] = np.inf, np.nan, -np.inf
    t, v = bf16(y)
    Q, S, QT, ST, sums = map(host, run_checkpoint(t, cols, "e4m3"))
    bad, bad_t = np.zeros((96, 3), bool), np.zeros((96, 3), bool)
    for r, c in ((3, 40), (50, 70), (70, 3)):
        bad[r, c // 32] = bad_t[c, r // 32] = True
    assert ((S[:, :3] == 255) == bad).all() and ((ST[:, :3] == 255) == bad_t).all()
    # The other blocks are as without them.
    P, R, PT, RT, _ = map(host, run_checkpoint(bf16(x)[0], cols, "e4m3"))
    assert (S[:, :3] == R[:, :3])[~bad].all() and (ST[:, :3] == RT[:, :3])[~bad_t].all()
    assert (Q == P)[~np.repeat(bad, 32, 1)].all() and (QT == PT)[~np.repeat(bad_t, 32, 1)].all()
    assert np.isinf(sums[40]) and np.isnan(sums[70]) and np.isinf(sums[3])


def test_checkpoint_sums_do_not_move():
    rows, cols = 5000, 200
    t, x = bf16(np.random.default_rng(3).normal(size=(rows, cols)) * 100)
    first = run_checkpoint(t, cols, "e4m3")
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, run_checkpoint(t, cols, "e4m3")))


def test_checkpoint_offsets_past_32_bits():
    rows, cols, ld = 70_000, 40, 1 << 16
    x = torch.empty((rows, ld), dtype=torch.bfloat16, device="cuda")
    v = torch.randn((rows, cols), device="cuda").to(torch.bfloat16)
    x[:, :cols] = v
    Q, S, QT, ST, sums = run_checkpoint(x, cols, "e4m3")
    wide = torch.zeros((rows, 64), dtype=torch.bfloat16, device="cuda")
    wide[:, :cols] = v
    want = run_checkpoint(wide, cols, "e4m3")
    assert all(torch.equal(a, b) for a, b in zip((Q, S, QT, ST, sums), want))
    n = rows // 32 * 32 - 64
    dr.check_codes(host(QT[:, n:].contiguous()), host(ST[:, n // 32:].contiguous()), host(v[n:].float()).T.copy(), 0, "e4m3")
    dr.check_codes(host(Q[-500:].contiguous()), host(S[-500:].contiguous()), host(v[-500:].float()), 0, "e4m3")


# ----------------------------------------------------------------- backward --


def run_backward(dh, Z, SZ, fmt_z, act, cols, fmt="e4m3", fmt_h="e4m3", dz=True, row=True, col=True, h=True, sums=True, pad=0, extra=2,
                 stream=None, dZ=None):
    rows = dh.shape[0]
    if dz and dZ is None:
        dZ = torch.full((rows, cols + pad), 777.0, dtype=torch.bfloat16, device="cuda")
    Q, S = (u8(rows, up32(cols) + pad), u8(rows, up32(cols) // 32 + extra, 0xDD)) if row else (None, None)
    QT, ST = (u8(cols, up32(rows) + pad), u8(cols, up32(rows) // 32 + extra, 0xDD)) if col else (None, None)
    HT, SHT = (u8(cols, up32(rows) + pad), u8(cols, up32(rows) // 32 + extra, 0xDD)) if h else (None, None)
    db = torch.full((cols,), float("nan"), device="cuda") if sums else None
    need = mx.mxfp8_checkpoint_workspace_size(rows, cols)
    ws = workspace(need)
    mx.mxfp8_act_backward(dZ if dz else None, dZ.stride(0) if dz else 0, Q, up32(cols) + pad, S, up32(cols) // 32 + extra, QT,
                          up32(rows) + pad, ST, up32(rows) // 32 + extra, HT, up32(rows) + pad, SHT, up32(rows) // 32 + extra, db, dh,
                          dh.stride(0), Z, Z.stride(0), SZ, SZ.stride(0), FMT[fmt_z], dr.ACTS.index(act), rows, cols, FMT[fmt], FMT[fmt_h],
                          ws, need, stream=stream)
    return dZ, Q, S, QT, ST, HT, SHT, db


def checkpoint_of(z, fmt):
    """z [rows, cols] in 8 bits, rubbish in the last block's free columns; the values."""
    rows, cols = z.shape
    wide = np.zeros((rows, up32(cols)))
    wide[:, :cols] = z
    c, s = ref.quantise(wide, fmt)
    v = ref.values(c, s, fmt)[:, :cols]
    c[:, cols:] = np.random.default_rng(0).integers(0, 256, size=(rows, up32(cols) - cols))
    return dev(c), dev(s), v


@pytest.mark.parametrize("act", dr.ACTS)
@pytest.mark.parametrize("fmt_z", ["e4m3", "e5m2"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_backward(rows, cols, fmt_z, act):
    rng = np.random.default_rng(rows + cols)
    Z, SZ, z = checkpoint_of(rng.normal(size=(rows, cols)) * 2, fmt_z)
    dh, g = bf16(rng.normal(size=(rows, cols)) * np.exp(rng.normal(size=(rows, 1))) * 1e-3, ld=-(-cols // 8) * 8 + 8)
    fmt, fmt_h = ("e5m2", "e4m3") if fmt_z == "e4m3" else ("e4m3", "e5m2")
    dZ, Q, S, QT, ST, HT, SHT, db = map(host, run_backward(dh, Z, SZ, fmt_z, act, cols, fmt, fmt_h, pad=16))
    h, slope, eh, es = dr.act(z, act)
    v, e = g * slope, np.abs(g) * es + 2 * EPS24 * np.abs(g * slope)
    dr.check_bf16(dZ[:, :cols], v, e, "dZ")
    assert (dZ[:, cols:] == 776.0).all()
    dr.check_codes(Q, S, v, e, fmt, "rows")
    dr.check_codes(QT, ST, v.T.copy(), e.T.copy(), fmt, "columns")
    dr.check_codes(HT, SHT, h.T.copy(), eh.T.copy(), fmt_h, "h")
    assert (np.abs(db - v.sum(0)) <= sum_bound(rows, v) + e.sum(0)).all()


def test_backward_outputs_alone_and_in_place():
    rows, cols = 300, 520
    rng = np.random.default_rng(5)
    Z, SZ, z = checkpoint_of(rng.normal(size=(rows, cols)), "e4m3")
    dh, _ = bf16(rng.normal(size=(rows, cols)))
    whole = run_backward(dh, Z, SZ, "e4m3", "gelu", cols)
    for only in ("dz", "row", "col", "h", "sums"):
        flags = {k: k == only for k in ("dz", "row", "col", "h", "sums")}
        for a, b in zip(whole, run_backward(dh, Z, SZ, "e4m3", "gelu", cols, **flags)):
            assert b is None or torch.equal(a, b)
    mine = dh.clone()
    again = run_backward(mine, Z, SZ, "e4m3", "gelu", cols, dZ=mine)
    assert all(torch.equal(a, b) for a, b in zip(whole, again))
    odd, _ = bf16(np.zeros((rows, cols)), ld=cols + 3, shift=1)
    assert torch.equal(run_backward(dh, Z, SZ, "e4m3", "gelu", cols, dZ=odd)[0], whole[0])


@pytest.mark.parametrize("act", dr.ACTS)
def test_backward_slope_against_differences(act):
    """The slope that the kernel uses is that of the activation it uses: h(z + s) - h(z - s) over 2 s
    between codes next to each other, by the mean value theorem within the slope's range there."""
    codes = np.arange(8, 120, dtype=np.uint8)                # positive codes, then their negatives
    for sign in (0, 0x80):
        c = (codes | sign)[None].repeat(32, 0)
        c = np.pad(c, ((0, 0), (0, up32(c.shape[1]) - c.shape[1])))
        cols = c.shape[1]
        s = np.full((32, cols // 32), 127 - 4, np.uint8)
        z = ref.values(c[:1], s[:1], "e4m3")[0]
        ones = torch.ones((32, cols), dtype=torch.bfloat16, device="cuda")
        db = host(run_backward(ones, dev(c), dev(s), "e4m3", act, cols)[-1]) / 32
        h, slope, eh, es = dr.act(z, act)
        assert (np.abs(db - slope) <= es + 80 * EPS24 * np.abs(slope)).all()
        n = 2.0 ** -10
        near = (dr.act(z + n, act)[0] - dr.act(z - n, act)[0]) / (2 * n)
        smooth = np.ones_like(z) if act != "relu" else (np.abs(z) > n)
        assert (np.abs(db - near) * smooth <= es + 80 * EPS24 + 2 * n * n * (1 + np.abs(z)) ** 3).all()


def test_backward_not_finite():
    rows, cols = 64, 96
    rng = np.random.default_rng(6)
    Z, SZ, z = checkpoint_of(rng.normal(size=(rows, cols)), "e4m3")
    SZ[5, 1] = 255                                           # a block of NaN
    dh, g = bf16(rng.normal(size=(rows, cols)))
    dh[40, 80] = float("inf")
    dZ, Q, S, QT, ST, HT, SHT, db = map(host, run_backward(dh, Z, SZ, "e4m3", "silu", cols))
    bad = np.zeros((rows, 3), bool)
    bad[5, 1] = bad[40, 2] = True
    assert ((S[:, :3] == 255) == bad).all()
    assert (ST[32:64, 0] == 255).all() and (ST[80, 1] == 255) and (ST == 255).sum() == 33
    assert (SHT[32:64, 0] == 255).all() and (SHT == 255).sum() == 32
    assert np.isnan(db[32:64]).all() and np.isinf(db[80]) and np.isfinite(np.delete(db, [*range(32, 64), 80])).all()


# --------------------------------------------------------------------- norm --

LENGTHS = [(1, 1), (3, 7), (1, 8192), (5, 32), (400, 100), (700, 256), (330, 257), (400, 1000), (350, 1001), (9, 1024), (400, 1024), (31, 1025),
           (330, 2048), (40, 4100), (5, 8192), (4, 8194), (3, 16384), (3, 16385), (2, 20000), (3, 32768), (700, 16)]


def norm_inputs(T, N, seed, mean=0.3):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(T, N)) * np.exp(rng.normal(size=(T, 1))) + mean * rng.normal(size=(T, 1))
    return rng, x


def check_norm(T, N, kind="bf16", w=True, b=True, ld=None, shift=0, eps=1e-5, stats=True, in_place=False, mean=0.3):
    rng, x = norm_inputs(T, N, T + N, mean)
    X, x = bf16(x, ld, shift)
    dw, w = param(rng.normal(size=N) + 1 if w else None, kind)
    db, b = param(rng.normal(size=N) if b else None, kind)
    w, b = (1.0 if w is None else w), (0.0 if b is None else b)
    Y = X if in_place else bf16(np.zeros((T, N)), ld, shift)[0]
    m, r = (torch.full((T,), float("nan"), device="cuda") for _ in range(2)) if stats else (None, None)
    mx.mxfp4_layer_norm(Y, Y.stride(0), m, r, X, X.stride(0), dw, db, KIND[kind], eps, T, N)
    y, mean, rstd, ey, em, er = dr.norm(x, w, b, eps)
    dr.check_bf16(host(Y), y, ey, "y")
    if stats:
        assert (np.abs(host(m) - mean) <= em + 2.0 ** -140).all() and (np.abs(host(r) - rstd) <= er).all()


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("T,N", LENGTHS)
def test_norm(T, N, kind):
    check_norm(T, N, kind)


@pytest.mark.parametrize("T,N", [(3, 64), (400, 100), (330, 1000), (5, 5000), (2, 20000)])
def test_norm_layouts(T, N):
    for shift in (0, 1, 2, 4):
        for pad in (0, 1, 2, 4, 8):
            check_norm(T, N, "fp32", ld=N + pad, shift=shift)
    check_norm(T, N, w=False)
    check_norm(T, N, b=False, stats=False)
    check_norm(T, N, in_place=True)
    check_norm(T, N, "fp32", w=False, b=False, eps=1.0)


# Enough rows for the streamed forms: 16-byte rows and others, one and several rows of a stage.
STREAMED = [(2500, 2056), (1300, 4104), (1250, 8192), (1300, 8190), (1280, 5001), (6500, 1032), (10000, 264), (10000, 513), (20000, 257)]


@pytest.mark.parametrize("T,N", STREAMED)
def test_norm_of_many_rows(T, N):
    check_norm(T, N, "fp32")
    check_norm(T, N, "bf16", ld=N + 1, shift=3, b=False)
    check_norm(T, N, w=False, in_place=True, stats=False, ld=N + 8 - N % 8)
    X, x = bf16(np.random.default_rng(0).normal(size=(T, N)))
    X[3, 5], X[T // 2, N - 1], X[T - 1, 0] = float("nan"), float("inf"), float("nan")
    Y = torch.empty_like(X)
    mx.mxfp4_layer_norm(Y, N, None, None, X, N, None, None, 0, 1e-5, T, N)
    bad = torch.isnan(Y)
    assert bad[[3, T // 2, T - 1]].all() and int(bad.sum()) == 3 * N


@pytest.mark.parametrize("T,N", STREAMED)
def test_norm_backward_of_many_rows(T, N):
    check_norm_backward(T, N, "fp32")
    check_norm_backward(T, N, "bf16", resid=False, ld=N + 1, shift=3)
    check_norm_backward(T, N, w=False, ld=N + 8 - N % 8, alias="x", params=(True, False))
    check_norm_backward(T, N, alias="dy", params=(False, True))
    check_norm_backward(T, N, alias="res")


def test_norm_rows_far_from_zero():
    """The variance is of differences from the mean, so a large mean costs no more than its own rounding."""
    check_norm(50, 4096, mean=1000.0)
    check_norm(1300, 4096, mean=1000.0)
    X, x = bf16(np.full((3, 777), 1.0) * [[2.5], [0.0], [-300.0]])
    Y, r = torch.empty_like(X), torch.empty(3, device="cuda")
    mx.mxfp4_layer_norm(Y, 777, None, r, X, 777, None, None, 0, 1e-5, 3, 777)
    assert (np.abs(host(Y)) <= 300 * 48 * EPS24 / np.sqrt(1e-5)).all() and (host(r) <= 1 / np.sqrt(1e-5) * (1 + 8 * EPS24)).all()


def test_norm_not_finite_stays_in_its_row():
    for T, N in ((20, 300), (400, 300), (20, 9000)):
        X, x = bf16(np.random.default_rng(0).normal(size=(T, N)))
        X[3, 5], X[7, 6] = float("nan"), float("inf")
        Y = torch.empty_like(X)
        mx.mxfp4_layer_norm(Y, N, None, None, X, N, None, None, 0, 1e-5, T, N)
        bad = np.isnan(host(Y))
        assert bad[[3, 7]].all() and bad.sum() == 2 * N


def check_norm_backward(T, N, kind="bf16", w=True, resid=True, ld=None, shift=0, params=(True, True), alias=None, stream=None):
    rng, x = norm_inputs(T, N, 3 * T + N)
    X, x = bf16(x, ld, shift)
    dY, dy = bf16(rng.normal(size=(T, N)) * 0.1, ld, shift)
    R, res = bf16(rng.normal(size=(T, N)) * 0.1, ld, shift) if resid else (None, 0.0)
    dw_, w = param(rng.normal(size=N) + 1 if w else None, kind)
    w = 1.0 if w is None else w
    _, mean, rstd, *_ = dr.norm(x, 1.0, 0.0, 1e-5)
    m, r = dev(mean.astype(np.float32)), dev(rstd.astype(np.float32))
    mean, rstd = host(m), host(r)
    dX = {"dy": dY, "x": X, "res": R, None: None}[alias]
    dX = bf16(np.zeros((T, N)), ld, shift)[0] if dX is None else dX
    dw, db = (torch.full((N,), float("nan"), device="cuda") if p else None for p in params)
    need = mx.mxfp4_layer_norm_workspace_size(T, N)
    ws = workspace(need)
    torch.cuda.synchronize()                                # (arrays are filled on the current stream)
    mx.mxfp4_layer_norm_backward(dX, dX.stride(0), dw, db, dY, dY.stride(0), X, X.stride(0), m, r, dw_, KIND[kind], R,
                                 R.stride(0) if resid else 0, T, N, ws, need, stream=stream)
    wx, ww, wb, ex, ew, eb = dr.norm_backward(x, dy, mean, rstd, w, res)
    dr.check_bf16(host(dX), wx, ex, "dx")
    for got, want, e in ((dw, ww, ew), (db, wb, eb)):
        if got is not None:
            assert (np.abs(host(got) - want) <= e + 2.0 ** -140).all()
    return dX, dw, db


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("T,N", LENGTHS + [(1300, 48), (3000, 1024), (1200, 2000), (700, 9000), (400, 17000)])
def test_norm_backward(T, N, kind):
    check_norm_backward(T, N, kind, resid=kind == "bf16")


@pytest.mark.parametrize("T,N", [(3, 64), (400, 100), (330, 1000), (5, 5000), (4, 12000), (2, 20000)])
def test_norm_backward_layouts(T, N):
    for shift in (0, 1, 2, 4):
        for pad in (0, 1, 4):
            check_norm_backward(T, N, "fp32", ld=N + pad, shift=shift)
    check_norm_backward(T, N, w=False)
    for params in ((True, False), (False, True), (False, False)):
        check_norm_backward(T, N, params=params)
    for alias in ("dy", "x", "res"):
        check_norm_backward(T, N, alias=alias)


def test_norm_backward_of_no_rows():
    dw, db = (torch.full((300,), float("nan"), device="cuda") for _ in range(2))
    mx.mxfp4_layer_norm_backward(None, 0, dw, db, None, 0, None, 0, None, None, None, 0, None, 0, 0, 300, None, 0)
    assert (host(dw) == 0).all() and (host(db) == 0).all()
    mx.mxfp4_layer_norm(None, 0, None, None, None, 0, None, None, 0, 1e-5, 0, 300)


def test_norm_backward_sums_do_not_move():
    first = check_norm_backward(2500, 1500)
    s = torch.cuda.Stream()
    for stream in (None, s):
        again = check_norm_backward(2500, 1500, stream=stream)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_norm_gradient_against_differences():
    """dx, dw and db against the definition's central differences in 64 bits."""
    T, N = 4, 48
    rng, x = norm_inputs(T, N, 1)
    X, x = bf16(x)
    dY, dy = bf16(rng.normal(size=(T, N)))
    dw_, w = param(rng.normal(size=N), "fp32")

    def loss(x, w, b):
        return (dr.norm(x, w, b, 1e-5)[0] * dy).sum()

    y, mean, rstd, *_ = dr.norm(x, w, 0.0, 1e-5)
    dX, dw, db = torch.empty_like(X), torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    ws = workspace(mx.mxfp4_layer_norm_workspace_size(T, N))
    mx.mxfp4_layer_norm_backward(dX, N, dw, db, dY, N, X, N, dev(mean.astype(np.float32)), dev(rstd.astype(np.float32)), dw_,
                                 mx.MXFP4_PARAM_FP32, None, 0, T, N, ws, ws.numel())
    n = 1e-5
    b = np.zeros(N)
    got = host(dX), host(dw), host(db)
    for i in range(N):
        e = np.zeros(N)
        e[i] = n
        for t in range(T):
            E = np.zeros((T, N))
            E[t, i] = n
            want = (loss(x + E, w, b) - loss(x - E, w, b)) / (2 * n)
            assert abs(got[0][t, i] - want) <= 2.0 ** -8 * abs(want) + 1e-5
        assert abs(got[1][i] - (loss(x, w + e, b) - loss(x, w - e, b)) / (2 * n)) <= 1e-5
        assert abs(got[2][i] - (loss(x, w, b + e) - loss(x, w, b - e)) / (2 * n)) <= 1e-5


def test_norm_rows_past_32_bits():
    T, N, ld = 70_000, 24, 1 << 16
    X = torch.empty((T, ld), dtype=torch.bfloat16, device="cuda")
    v = torch.randn((T, N), device="cuda").to(torch.bfloat16)
    X[:, :N] = v
    Y = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    m, r = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    mx.mxfp4_layer_norm(Y, N, m, r, X, ld, None, None, 0, 1e-5, T, N)
    y, _, _, ey, *_ = dr.norm(host(v[-300:].float()), 1.0, 0.0, 1e-5)
    dr.check_bf16(host(Y[-300:]), y, ey)
    out = []
    ws = workspace(mx.mxfp4_layer_norm_workspace_size(T, N))
    for x, l in ((X, ld), (v, N)):
        dX, dw, db = torch.empty_like(v), torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
        mx.mxfp4_layer_norm_backward(dX, N, dw, db, Y, N, x, l, m, r, None, 0, None, 0, T, N, ws, ws.numel())
        out.append((dX, dw, db))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*out))


def test_operators_in_a_graph():
    """A norm, a checkpoint and their backward passes captured together, replayed on new inputs, two
    graphs with workspaces of their own in turn."""
    T, N = 200, 640

    def captured(seed):
        rng = np.random.default_rng(seed)
        X, x = bf16(rng.normal(size=(T, N)))
        Z, SZ, z = checkpoint_of(rng.normal(size=(T, N)), "e4m3")
        Y, dX = torch.empty_like(X), torch.empty_like(X)
        m, r, dw, db = (torch.empty(n, device="cuda") for n in (T, T, N, N))
        ws = workspace(max(mx.mxfp4_layer_norm_workspace_size(T, N), mx.mxfp8_checkpoint_workspace_size(T, N)))
        Q, S, QT, ST, sums = u8(T, N), u8(T, N // 32), u8(N, up32(T)), u8(N, up32(T) // 32), torch.empty(N, device="cuda")

        def calls():
            mx.mxfp4_layer_norm(Y, N, m, r, X, N, None, None, 0, 1e-5, T, N)
            mx.mxfp4_layer_norm_backward(dX, N, dw, db, Y, N, X, N, m, r, None, 0, Y, N, T, N, ws, ws.numel())
            mx.mxfp8_act_backward(dX, N, Q, N, S, N // 32, None, 0, None, 0, None, 0, None, 0, None, dX, N, Z, N, SZ, N // 32, 0, 2, T, N, 0,
                                  0, None, 0)
            mx.mxfp8_checkpoint(None, 0, None, 0, QT, up32(T), ST, up32(T) // 32, sums, dX, N, T, N, 0, ws, ws.numel())
        calls()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            calls()
        return g, calls, X, (Y, dX, m, r, dw, db, Q, S, QT, ST, sums)

    graphs = [captured(seed) for seed in (1, 2)]
    for k in range(4):
        for g, calls, X, outs in graphs:
            X.normal_()
            g.replay()
        torch.cuda.synchronize()
        for g, calls, X, outs in graphs:
            got = [t.clone() for t in outs]
            calls()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, outs))
