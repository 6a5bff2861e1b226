"""Expert-layer operators on the GPU through the C ABI against plain 64-bit
forms (tests/expert_ref.py).

Bounds, derived from the arithmetic:
  product   |D - ref| <= ulp_bf16(ref) + 2^-20 sum |a b|: one bf16 rounding and
            fp32 accumulation, as for the dense GEMMs.
  gated     with dg, du = 2^-20 sum |a b| of the two products, |silu'| <= 1.1
            and a few ulp of exp, divide and multiply, h lies within
            1.1 |u| dg + |silu(g)| du + 1.1 dg du + 2^-19 (1 + |g|) |h| of the
            exact value; the scale has to be that of some amax inside the
            block's interval, and each code that of some h inside its own
            (the rounding is monotonic).
  gates     expf is good to 2 ulp, the sums add at most E rounded terms of one
            sign in chains of E / 32 + 5, one divide: (E / 32 + 16) 2^-23.
  join      ulp_bf16(ref) + 2^-18 of the terms' magnitudes: chains of at most
            k + 3 roundings, and two norms whose sums of squares add 2^-20.
Integers and the codes of exact inputs are equal.
"""
import numpy as np
import pytest

import block_scaled_mxfp4_gb300 as mx
import expert_ref as ref
from parity_util import bf16_bits_to_f64, d_to_bits, ulp_bf16

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


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


def bf16(x):
    """float64 -> (bf16 tensor on the GPU, its values)."""
    t = torch.from_numpy(np.asarray(x, np.float64)).to(torch.bfloat16)
    return t.cuda(), t.double().numpy()


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


# ------------------------------------------------------------------ routing --


def run_route(logits, k, mode, mask=None, scale=1.0, ldl=None, stream=None, fill=-7):
    T, E = logits.shape
    if ldl is not None:
        wide = torch.full((max(T, 1), ldl), 100.0, dtype=logits.dtype, device="cuda")
        wide[:T, :E] = logits
        logits = wide
    i32 = dict(dtype=torch.int32, device="cuda")
    ids, slot_row = torch.full((T, k), fill, **i32), torch.full((T, k), fill, **i32)
    offsets, row_token = torch.full((E + 1,), fill, **i32), torch.full((T * k,), fill, **i32)
    gates = torch.full((T, k), float("nan"), device="cuda")
    need = mx.mxfp4_moe_route_workspace_size(T, E)
    ws = torch.full((max(need, 256),), 0xAB, dtype=torch.uint8, device="cuda")
    kind = mx.MXFP4_LOGITS_FP32 if logits.dtype == torch.float32 else mx.MXFP4_LOGITS_BF16
    mx.mxfp4_moe_route(ids, gates, offsets, row_token, slot_row, logits, logits.stride(0) if T else E, kind,
                       mask, T, E, k, mode, scale, ws, need, stream)
    return [host(v) for v in (ids, gates, offsets, row_token, slot_row)]


def check_route(logits, k, mode, mask=None, **kw):
    got = run_route(logits, k, mode, None if mask is None else dev(mask), **kw)
    x = logits.double().cpu().numpy()
    E = x.shape[1]
    ids, gates = ref.route(x, k, mode, mask)
    offsets, row_token, slot_row = ref.grouping(ids, E)
    np.testing.assert_array_equal(got[0], ids)
    np.testing.assert_array_equal(got[2], offsets)
    np.testing.assert_array_equal(got[3], row_token)
    np.testing.assert_array_equal(got[4], slot_row)
    np.testing.assert_allclose(got[1], gates * kw.get("scale", 1.0), rtol=(E / 32 + 16) * 2.0 ** -23, atol=1e-37)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 128, 8), (3, 5, 5), (17, 33, 4), (64, 64, 16), (65, 64, 2),
                                   (127, 257, 8), (300, 512, 6), (1000, 96, 8), (130, 1024, 3)])
@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_route(T, E, k, mode, dtype):
    g = torch.Generator().manual_seed(T * E + k)
    x = torch.randn((T, E), generator=g) * 2
    x = x.to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()
    check_route(x, k, mode)


def test_route_of_no_tokens():
    got = run_route(torch.empty((0, 9), device="cuda"), 3, 0)
    np.testing.assert_array_equal(got[2], np.zeros(10, np.int32))


@pytest.mark.parametrize("T", [40, 500])
def test_route_ties_go_to_the_lowest_index(T):
    g = torch.Generator().manual_seed(3)
    x = torch.randint(-1, 2, (T, 70), generator=g).float()
    x[0] = 0.0
    x[1, ::2] = -0.0                                       # -0 and 0 are equal
    check_route(x.cuda(), 9, 0)
    check_route(x.to(torch.bfloat16).cuda(), 9, 1)


@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("T", [30, 400])
def test_route_masked_rows_and_strange_logits(T, mode):
    rng = np.random.default_rng(T)
    x = rng.normal(size=(T, 40)).astype(np.float32)
    x[2] = -np.inf                                         # nothing left
    x[3, 5:] = -np.inf                                     # fewer than k left
    x[4, 7] = np.nan
    x[5] = np.nan
    x[6, [3, 9]] = np.inf                                  # share the softmax
    x[7] = np.finfo(np.float32).min                        # the type's lowest value is a value
    x[8, 1:] = np.finfo(np.float32).min
    x[9] = -1e30
    mask = (rng.uniform(size=T) < 0.7).astype(np.uint8)
    mask[:10] = 1
    check_route(dev(x), 8, mode, mask)
    check_route(dev(x), 8, mode, np.zeros(T, np.uint8))    # every token masked


def test_route_strided_scaled_and_all_to_one():
    g = torch.Generator().manual_seed(5)
    x = torch.randn((200, 24), generator=g).cuda()
    check_route(x, 4, 0, ldl=31, scale=2.5)
    x[:, 1:] -= 100
    check_route(x, 1, 0)


@pytest.mark.parametrize("T,E,k", [(10, 200, 8), (16, 400, 5), (13, 900, 8), (9, 100, 9), (9, 200, 10), (9, 500, 16), (9, 1000, 12),
                                   (20, 128, 8), (56, 16, 4), (33, 600, 8)])
def test_route_few_tokens(T, E, k):
    g = torch.Generator().manual_seed(T + E)
    x = torch.randn((T, E), generator=g) * 2
    check_route(x.cuda(), k, 1)
    check_route(x.to(torch.bfloat16).cuda(), k, 0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,E,k,mode", [(80001, 8, 2, 0), (78000, 30, 8, 1), (40001, 64, 4, 0), (20000, 100, 8, 1),
                                        (9985, 250, 8, 2), (5000, 512, 6, 0), (2500, 777, 7, 1), (20000, 128, 12, 0),
                                        (5000, 251, 5, 1), (30000, 12, 10, 1), (20000, 64, 9, 0), (12000, 256, 16, 1),
                                        (1000, 100, 9, 2), (1000, 200, 10, 0), (1000, 512, 11, 1), (500, 1024, 15, 0)])
def test_route_many_tokens(T, E, k, mode, dtype):
    """The forms for many tokens, all lane counts: random logits, then ties,
    masked tokens, infinities and NaN among them."""
    g = torch.Generator().manual_seed(T + E)
    x = torch.randn((T, E), generator=g) * 2
    x[: T // 2] = torch.round(x[: T // 2])                 # many ties
    x[5::97] = float("-inf")
    x[6::101, 1:] = float("-inf")
    x[7::103, E // 2] = float("nan")
    x[8::107, E // 3] = float("inf")
    x[9::109, ::2] = -0.0
    x[10::113] = -3e38
    x = x.to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()
    mask = (np.random.default_rng(T).uniform(size=T) < 0.9).astype(np.uint8)
    got = run_route(x, k, mode, dev(mask), ldl=E + 3 if mode == 1 else None)
    want = ref.route_many(x.double().cpu().numpy(), k, mode, mask)
    for i, what in enumerate(("ids", "gates", "offsets", "row_token", "slot_row")):
        if what == "gates":
            np.testing.assert_allclose(got[1], want[1], rtol=(E / 32 + 16) * 2.0 ** -23, atol=1e-37)
        else:
            np.testing.assert_array_equal(got[i], want[i], err_msg=what)


def test_the_plain_forms_of_routing_agree():
    x = np.round(np.random.default_rng(0).normal(size=(90, 17)) * 2)
    x[3] = -np.inf
    x[4, 5] = np.nan
    for mode in (0, 1, 2):
        ids, gates = ref.route(x, 6, mode)
        many = ref.route_many(x, 6, mode)
        np.testing.assert_array_equal(ids, many[0])
        np.testing.assert_allclose(gates, many[1], rtol=1e-12)
        for u, v in zip(ref.grouping(ids, 17), many[2:]):
            np.testing.assert_array_equal(u, v)


# ---------------------------------------------------------------- quantiser --


def run_quantize(fmt, x, K, slot_row, ids, offsets, groups, rows, ldq=None, k=None):
    packed = fmt == "e2m1"
    ldq = ldq or -(-K // 32) * 32
    Q = torch.full((max(rows, 1), ldq // 2 if packed else ldq), 0xEE, dtype=torch.uint8, device="cuda")
    S = torch.full((mx.mxfp4_group_scale_size(rows, groups, K),), 0xDD, dtype=torch.uint8, device="cuda")
    T = x.shape[0]
    k = k or (1 if slot_row is None else slot_row.shape[1])
    args = (Q, ldq, S, x, x.stride(0), T, K, None if slot_row is None else dev(slot_row),
            None if ids is None else dev(ids), k, dev(offsets), groups, rows)
    if packed:
        mx.mxfp4_group_quantize(*args)
    else:
        mx.mxfp8_group_quantize(*args, {"e4m3": mx.MXFP8_E4M3, "e5m2": mx.MXFP8_E5M2}[fmt])
    return host(Q), host(S)


def random_ids(T, E, k, seed, skip=0.0):
    rng = np.random.default_rng(seed)
    ids = np.argsort(rng.uniform(size=(T, E)) + np.linspace(0, 1, E), axis=1)[:, :k].astype(np.int32)
    ids[rng.uniform(size=(T, k)) < skip] = -1
    return ids


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3", "e5m2"])
@pytest.mark.parametrize("T,E,k,K,skip", [(1, 4, 2, 32, 0), (1, 4, 4, 256, 0), (40, 3, 3, 96, 0.3), (300, 5, 2, 288, 0.1),
                                          (129, 2, 1, 1056, 0), (7, 64, 6, 544, 0.5)])
def test_group_quantize(fmt, T, E, k, K, skip):
    rng = np.random.default_rng(T + K)
    ids = random_ids(T, E, k, T, skip)
    offsets, row_token, slot_row = ref.grouping(ids, E)
    x, xv = bf16(rng.normal(size=(T, K)) * np.exp(rng.normal(size=(T, K)) * 2))
    xv = xv.copy()
    if T > 3:
        x[1] = 0
        xv[1] = 0
        x[2, :32] = -0.0
        xv[2, :32] = -0.0
    Q, S = run_quantize(fmt, x, K, slot_row, ids, offsets, E, T * k)
    codes, scales = ref.quantise(xv, fmt)
    n = offsets[-1]
    w = codes.shape[1]
    np.testing.assert_array_equal(Q[:n, :w], codes[row_token[:n]])
    np.testing.assert_array_equal(S[ref.scale_places(offsets, K)], scales[row_token[:n]])
    assert (Q[n:] == 0xEE).all()                           # rows of no group stay
    if (K // 32) % 2 and n:
        assert (S[ref.scale_places(offsets, K)[:, -1] + 1] == 0x7F).all()


def test_group_quantize_in_place_rows_strides_and_specials():
    """Already grouped rows (no slots), wider strides, empty groups, a capacity above the rows."""
    offsets = np.array([0, 0, 5, 5, 140, 141, 141], np.int32)
    rows, K = 150, 160
    rng = np.random.default_rng(9)
    wide = rng.normal(size=(rows, K + 24))
    wide[3, 40] = np.inf
    wide[4, 0] = np.nan
    wide[6, 64:96] = 3.0e38
    wide[7, 64:96] = 1e-39                                 # bf16 subnormals
    t, v = bf16(wide)
    Q, S = run_quantize("e2m1", t[:, :K], K, None, None, offsets, 6, rows, ldq=192)
    v = v[:, :K].copy()
    bad = ~np.isfinite(v.reshape(rows, -1, 32)).all(-1)
    assert bad.sum() == 2
    codes, scales = ref.quantise(np.where(np.isfinite(v), v, 0), "e2m1")
    at = ref.scale_places(offsets, K)
    fine = np.repeat(~bad, 16, axis=1)
    n = offsets[-1]
    np.testing.assert_array_equal(np.where(fine, Q[:, :K // 2], 0)[:n], np.where(fine, codes, 0)[:n])
    np.testing.assert_array_equal(S[at], np.where(bad, 255, scales)[:n])
    assert (Q[n:] == 0xEE).all() and (Q[:n, K // 2:] == 0xEE).all()


def test_group_quantize_skips_rows_outside_the_arrays():
    """Slots whose row or expert cannot be are left out rather than followed."""
    ids = np.array([[0, 1], [5, -1], [1, 0]], np.int32)
    slot_row = np.array([[0, 99], [2, 1], [3, -3]], np.int32)
    offsets = np.array([0, 2, 4], np.int32)
    x, v = bf16(np.ones((3, 64)))
    Q, S = run_quantize("e2m1", x, 64, slot_row, ids, offsets, 2, 4)
    written = (Q != 0xEE).any(1)
    np.testing.assert_array_equal(written, [True, False, False, True])


# ----------------------------------------------------------------- products --

FMT_CODE = {"e2m1": None, "e4m3": 0, "e5m2": 1, "e2m3": mx.MXFP6_E2M3, "e3m2": mx.MXFP6_E3M2,
            "e2m1 padded": mx.MXFP4_E2M1_PADDED}


def random_operand(rng, rows, K, fmt, spread=2):
    if fmt == "e2m1":
        q = rng.integers(0, 256, size=(rows, K // 2), dtype=np.uint8)
    elif fmt in ref.PADDED:
        q = rng.integers(0, 256, size=(rows, K), dtype=np.uint8)   # the padding bytes too: nothing reads them
    else:
        top = {"e4m3": 0x70, "e5m2": 0x50}[fmt]
        q = (rng.integers(0x20, top, size=(rows, K)) | rng.integers(0, 2, size=(rows, K)) << 7).astype(np.uint8)
    return q, rng.integers(127 - spread, 128 + spread, size=(rows, K // 32)).astype(np.uint8)


class Grouped:
    """Operands of one grouped product on the GPU and their values."""

    def __init__(self, counts, N, K, fmt="e2m1", fmt_b=None, halves=1, seed=0, capacity=0, pad_k=0, spread=2):
        rng = np.random.default_rng(seed)
        fmt_b = fmt_b or fmt
        self.fmt, self.fmt_b, self.N, self.K, self.E = fmt, fmt_b, N, K, len(counts)
        self.offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        n = int(self.offsets[-1])
        self.rows = n + capacity
        q, s = random_operand(rng, self.rows, K, fmt, spread)
        self.A = ref.values(q, s, fmt)
        bq, bs = zip(*[random_operand(rng, halves * N, K, fmt_b, spread) for _ in range(self.E)])
        self.B = np.stack([ref.values(a, b, fmt_b) for a, b in zip(bq, bs)])
        self.qA, self.sA, self.qB = q, s, np.stack(bq)
        self.lda = K + pad_k
        self.ldb = K + pad_k
        wide = lambda m, d: np.concatenate([m, np.full((*m.shape[:-1], pad_k // d), 0xFF, np.uint8)], -1)
        self.dA = dev(wide(q, 2 if fmt == "e2m1" else 1))
        self.dB = dev(wide(self.qB, 2 if fmt_b == "e2m1" else 1))
        # Scales of what is not there are NaN: nothing may come from them.
        self.dSA = dev(ref.grouped_scales(s, self.offsets, K, self.rows, fill=255))
        self.dSB = dev(np.concatenate([ref.relaid(b[h * N:(h + 1) * N], K) for b in bs for h in range(halves)]))
        self.dO = dev(self.offsets)

    def workspace(self):
        need = mx.mxfp4_grouped_workspace_size(self.rows, self.E, self.N, self.K)
        return torch.full((max(need, 256),), 0xA5, dtype=torch.uint8, device="cuda"), need

    def gemm(self, alpha=1.0, ldd=None, stream=None, out=None, ws=None):
        ldd = ldd or self.N
        D = out if out is not None else torch.full((max(self.rows, 1), ldd), 7.0, dtype=torch.bfloat16, device="cuda")
        ws, need = ws or self.workspace()
        args = (D, ldd, self.dA, self.lda, self.dSA, self.dB, self.ldb, self.N * self.ldb, self.dSB, self.dO, self.E,
                self.rows, self.N, self.K)
        if self.fmt == "e2m1":
            mx.mxfp4_grouped_gemm(*args, alpha, ws, need, stream)
        else:
            mx.mxfp8_grouped_gemm(*args, FMT_CODE[self.fmt], FMT_CODE[self.fmt_b], alpha, ws, need, stream)
        return D

    def swiglu(self, fmt_h="e2m1", alpha=1.0, ldh=None, stream=None):
        F = self.N
        ldh = ldh or F
        H = torch.full((max(self.rows, 1), ldh // 2 if fmt_h == "e2m1" else ldh), 0xEE, dtype=torch.uint8, device="cuda")
        SH = torch.full((mx.mxfp4_group_scale_size(self.rows, self.E, F),), 0xDD, dtype=torch.uint8, device="cuda")
        ws, need = self.workspace()
        args = (H, ldh, SH, self.dA, self.lda, self.dSA, self.dB, self.ldb, 2 * F * self.ldb, self.dSB, self.dO, self.E,
                self.rows, F, self.K)
        if self.fmt == "e2m1":
            mx.mxfp4_grouped_swiglu(*args, alpha, ws, need, stream)
        else:
            mx.mxfp8_grouped_swiglu(*args, FMT_CODE[self.fmt], FMT_CODE[self.fmt_b], FMT_CODE[fmt_h], alpha, ws, need,
                                    stream)
        return H, SH


def check_gemm(p, alpha=1.0, ldd=None):
    D = p.gemm(alpha, ldd)
    torch.cuda.synchronize()
    got = bf16_bits_to_f64(d_to_bits(D))
    want, mag = ref.product(p.A, p.B, p.offsets)
    want, mag = alpha * want, abs(alpha) * mag
    n = p.offsets[-1]
    err = np.abs(got[:n, :p.N] - want[:n])
    bound = ulp_bf16(want[:n]) + 2.0 ** -20 * mag[:n]
    assert np.isfinite(got[:n, :p.N]).all()
    assert (err <= bound).all(), (np.argwhere(err > bound)[:8], (err / bound).max())
    assert (got[n:] == 7.0).all() and (got[:, p.N:] == 7.0).all()      # nothing else is written


COUNTS = {
    "one row": [1],
    "one row of many": [0, 0, 1, 0],
    "decode": [2, 0, 1, 1, 0, 3, 1, 0],
    "tile edges": [255, 256, 257, 0, 128, 129, 127],
    "ragged": [13, 400, 0, 0, 71, 1, 290],
    "empty ends": [0, 0, 30, 0],
}


@pytest.mark.parametrize("name", sorted(COUNTS))
@pytest.mark.parametrize("N,K", [(256, 256), (320, 96), (40, 800), (1, 32), (515, 1056)])
def test_grouped_gemm(name, N, K):
    check_gemm(Grouped(COUNTS[name], N, K, seed=N + K))


@pytest.mark.parametrize("fmt,fmt_b", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2")])
@pytest.mark.parametrize("name,N,K", [("decode", 256, 256), ("tile edges", 320, 96), ("ragged", 72, 800), ("one row", 8, 32)])
def test_grouped_gemm_bytes(fmt, fmt_b, name, N, K):
    check_gemm(Grouped(COUNTS[name], N, K, fmt, fmt_b, seed=N + K))


@pytest.mark.parametrize("fmt,fmt_b", [("e2m3", "e2m3"), ("e3m2", "e4m3"), ("e5m2", "e2m1 padded"), ("e2m1 padded", "e3m2")])
@pytest.mark.parametrize("name,N,K", [("decode", 72, 288), ("ragged", 256, 160)])
def test_grouped_products_of_padded_formats(fmt, fmt_b, name, N, K):
    check_gemm(Grouped(COUNTS[name], N, K, fmt, fmt_b, seed=N + K))
    p = Grouped(COUNTS[name], 96, K, fmt, fmt_b, halves=2, seed=N + K)
    check_swiglu(p, "e4m3", small(p))


def test_grouped_gemm_strides_alpha_capacity():
    check_gemm(Grouped(COUNTS["ragged"], 264, 320, capacity=300, pad_k=64), alpha=-0.375, ldd=280)
    check_gemm(Grouped(COUNTS["decode"], 33, 320, capacity=1, pad_k=32), alpha=2.0, ldd=35)


def test_grouped_gemm_without_rows():
    p = Grouped([0, 0, 0], 64, 64, capacity=5)
    D = p.gemm()
    torch.cuda.synchronize()
    assert (D == 7.0).all()
    mx.mxfp4_grouped_gemm(D, 64, p.dA, 64, p.dSA, p.dB, 64, 64 * 64, p.dSB, p.dO, 3, 0, 64, 64, 1.0, None, 0)


def test_grouped_gemm_many_tiles_and_many_groups():
    """Several tiles per CTA pair, and more groups than one warp's prefix sum."""
    check_gemm(Grouped([600, 0, 300], 4200, 512, seed=2))
    rng = np.random.default_rng(4)
    check_gemm(Grouped(rng.integers(0, 4, size=700).tolist(), 48, 64, seed=3))
    check_gemm(Grouped(([0] * 1023) + [3], 16, 32, seed=3))


@pytest.mark.parametrize("counts,N,K", [([1], 256, 4096), ([3, 2], 300, 8192), ([40], 512, 4096), ([200, 90], 700, 2048),
                                        ([300], 2000, 1504), ([1] * 8, 4096, 1024), ([256] * 5, 4352, 1024)])
def test_grouped_gemm_few_tiles_long_k(counts, N, K):
    """Fewer tiles than CTA pairs (or an uneven number of them), long reductions."""
    check_gemm(Grouped(counts, N, K, seed=K, spread=1))


# Rows per group on either side of the kernels' forms: at most 32 in all, 112 a
# group on average (with groups of more among them), above; tables of every size.
FORMS = {
    "32 rows": [0, 31, 1], "33 rows": [0, 32, 1], "small groups": [1, 130, 60, 0, 300, 20, 7, 128], "112 a group": [256, 0, 65, 127],
    "larger": [257, 0, 129, 127], "81 groups": [3] * 80 + [200], "861 groups": [1] * 860 + [300], "861 larger": [0] * 860 + [128 * 861 // 8, 5],
}


@pytest.mark.parametrize("name", sorted(FORMS))
def test_grouped_products_of_every_form(name):
    counts, few = FORMS[name], len(FORMS[name]) > 100
    N, K = (24, 64) if few else (392, 672)
    capacity = 128 * len(counts) if name == "861 larger" else 0
    check_gemm(Grouped(counts, N, K, seed=1, capacity=capacity))
    check_gemm(Grouped(counts, N + 1, K, "e4m3", "e5m2", seed=2, capacity=capacity))
    for fmt, fmt_h in (("e2m1", "e2m1"), ("e4m3", "e4m3"), ("e5m2", "e5m2")):
        p = Grouped(counts, 32 if few else 224, K, fmt, halves=2, seed=3, capacity=capacity)
        check_swiglu(p, fmt_h, 0.01)


@pytest.mark.parametrize("counts,N", [([40, 130, 7, 0, 64, 1], 3600), ([3, 1, 2, 4, 1, 5], 3601), ([40, 9, 0, 130] * 4, 3400),
                                      ([2, 0, 3, 1] * 5, 2700)])
def test_grouped_products_in_rounds_of_small_groups(counts, N):
    """More tiles than half of the SMs, or than all of them: nothing is halved."""
    check_gemm(Grouped(counts, N, 416, seed=N))
    for fmt, fmt_h in (("e2m1", "e2m1"), ("e4m3", "e5m2")):
        p = Grouped(counts, N // 64 * 32, 416, fmt, halves=2, seed=N)
        check_swiglu(p, fmt_h, 0.01)


def test_grouped_gemm_repeats_bit_for_bit_and_shares_a_workspace():
    a = Grouped([5, 0, 130], 520, 4096, seed=1)
    b = Grouped([2, 2], 300, 2048, seed=2)
    size = max(a.workspace()[1], b.workspace()[1])
    ws = (torch.full((max(size, 256),), 0x5A, dtype=torch.uint8, device="cuda"), size)
    first = [d_to_bits(p.gemm(ws=ws)).copy() for p in (a, b)]
    outs = [[p.gemm(ws=ws) for p in (a, b)] for _ in range(6)]
    torch.cuda.synchronize()
    for pair in outs:
        for got, want in zip(pair, first):
            np.testing.assert_array_equal(d_to_bits(got), want)


def test_grouped_products_in_a_graph_and_on_a_side_stream():
    p = Grouped([5, 0, 130], 520, 2048, seed=1)
    want = d_to_bits(p.gemm()).copy()
    D = torch.zeros((p.rows, p.N), dtype=torch.bfloat16, device="cuda")
    ws = p.workspace()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        p.gemm(out=D, ws=ws)
    for _ in range(3):
        D.zero_()
        graph.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(d_to_bits(D), want)
    # New offsets in the same buffer count at the next replay.
    p.dO.copy_(dev(np.array([0, 0, 135, 135], np.int32)))
    p.dSA.copy_(dev(ref.grouped_scales(p.sA, np.array([0, 0, 135, 135]), p.K, p.rows)))
    graph.replay()
    torch.cuda.synchronize()
    other, mag = ref.product(p.A, p.B, [0, 0, 135, 135])
    got = bf16_bits_to_f64(d_to_bits(D))
    assert (np.abs(got - other) <= ulp_bf16(other) + 2.0 ** -20 * mag).all()
    with torch.cuda.stream(side):
        D2 = p.gemm(stream=side)
    side.synchronize()
    np.testing.assert_array_equal(d_to_bits(D2), d_to_bits(D))


def test_grouped_gemm_nan_scales_stay_in_their_row():
    p = Grouped([4, 140], 64, 256)
    at = ref.scale_places(p.offsets, p.K)
    s = p.dSA.clone()
    s[dev(at[[1, 100], 3])] = 255
    p.dSA = s
    D = host(p.gemm().float())
    bad = np.isnan(D).any(1)
    assert np.isnan(D[[1, 100]]).all() and bad.sum() == 2


def test_grouped_gemm_ignores_offsets_out_of_order():
    """Unordered or oversized offsets give unspecified values and no access outside."""
    p = Grouped([10, 10, 10], 64, 64)
    for bad in ([0, 50, 20, 30], [-5, 10, 9000, 12], [3, 2, 1, 0]):
        p.dO = dev(np.array(bad, np.int32))
        p.gemm()
    torch.cuda.synchronize()


# -------------------------------------------------------------------- gated --


def check_swiglu(p, fmt_h, alpha=1.0, ldh=None):
    H, SH = p.swiglu(fmt_h, alpha, ldh)
    H, SH = host(H), host(SH)
    F, n = p.N, p.offsets[-1]
    gu, mag = ref.product(p.A, p.B, p.offsets)
    gu, mag = alpha * gu[:n], abs(alpha) * mag[:n] * 2.0 ** -20
    g, u, dg, du = gu[:, :F], gu[:, F:], mag[:, :F], mag[:, F:]
    silu = g / (1 + np.exp(-g))
    h = silu * u
    d = 1.1 * np.abs(u) * dg + np.abs(silu) * du + 1.1 * dg * du + 2.0 ** -19 * (1 + np.abs(g)) * np.abs(h) + 1e-38
    scales = SH[ref.scale_places(p.offsets, F)].astype(int)
    lo, hi = (np.abs(h) - d).clip(0).reshape(n, -1, 32).max(-1), (np.abs(h) + d).reshape(n, -1, 32).max(-1)
    ex = np.vectorize(lambda v: ref.scale_exponent(v, fmt_h), otypes=[int])
    s = scales - 127
    low = np.where(lo == 0, -127, ex(lo))                  # from 0 on: any small amax, or none at all (s = 0)
    assert ((low <= s) & (s <= ex(hi)) | (lo == 0) & (s == 0)).all()
    width = F // 2 if fmt_h == "e2m1" else F
    got = ref.values(H[:n, :width], scales.astype(np.uint8), fmt_h)
    per = np.repeat(s, 32, axis=1)

    def rounded(v):
        c, neg = ref.to_codes(np.ldexp(v, -per), fmt_h)
        return np.ldexp(ref.GRIDS[fmt_h][c] * np.where(neg, -1, 1), per)

    assert ((rounded(h - d) <= got) & (got <= rounded(h + d))).all()
    assert (H[n:] == 0xEE).all() and (H[:, width:] == 0xEE).all()
    if (F // 32) % 2 and n:
        assert (SH[ref.scale_places(p.offsets, F)[:, -1] + 1] == 0x7F).all()


def small(p):
    """alpha that brings the products to the activation's interesting range."""
    return float(2.0 ** -np.round(np.log2(np.abs(p.A[:1] @ p.B[0].T).mean() + 1e-9)))


@pytest.mark.parametrize("name", sorted(COUNTS))
@pytest.mark.parametrize("F,K", [(128, 256), (32, 96), (160, 800), (352, 1056)])
def test_grouped_swiglu(name, F, K):
    p = Grouped(COUNTS[name], F, K, halves=2, seed=F + K)
    check_swiglu(p, "e2m1", small(p))


@pytest.mark.parametrize("fmt_h", ["e4m3", "e5m2"])
@pytest.mark.parametrize("name,F,K", [("decode", 128, 256), ("tile edges", 96, 96), ("ragged", 288, 800)])
def test_grouped_swiglu_bytes(fmt_h, name, F, K):
    p = Grouped(COUNTS[name], F, K, "e4m3", halves=2, seed=F + K)
    check_swiglu(p, fmt_h, small(p))


def test_grouped_swiglu_strides_and_capacity():
    p = Grouped(COUNTS["ragged"], 160, 320, halves=2, capacity=300, pad_k=64)
    check_swiglu(p, "e2m1", small(p), ldh=224)


@pytest.mark.parametrize("counts,F,K", [([1], 256, 4096), ([40, 3], 96, 4096), ([300], 1024, 2048), ([256] * 5, 2176, 1024)])
def test_grouped_swiglu_few_tiles_long_k(counts, F, K):
    p = Grouped(counts, F, K, halves=2, seed=K, spread=1)
    check_swiglu(p, "e2m1", small(p))


def test_grouped_swiglu_extreme_gates():
    """Large products of either sign: silu goes to g or to 0, no overflow on the way."""
    p = Grouped([40], 64, 64, halves=2, seed=8)
    check_swiglu(p, "e2m1", small(p) * 256)
    check_swiglu(p, "e2m1", small(p) * 2.0 ** -60)


def test_grouped_swiglu_marks_blocks_that_are_not_finite():
    p = Grouped([6], 64, 64, halves=2, seed=8)
    s = p.dSA.clone()
    s[dev(ref.scale_places(p.offsets, p.K)[2])] = 255       # row 2: NaN throughout
    p.dSA = s
    H, SH = p.swiglu("e2m1", small(p))
    got = host(SH)[ref.scale_places(p.offsets, 64)]
    assert (got[2] == 255).all() and (np.delete(got, 2, 0) != 255).all()


# --------------------------------------------------------------------- join --


def check_combine(T, k, N, rows=None, post=True, pre=True, resid=True, norm=True, h_out=True, pad=0, slots=True,
                  skip=0.0, offset=0, seed=0):
    rng = np.random.default_rng(seed + T + N)
    rows = rows or max(T * k, 1)
    slot = rng.permutation(rows)[:T * k].reshape(T, k).astype(np.int32) if slots else None
    if slots:
        slot[rng.uniform(size=slot.shape) < skip] = -1
        if T > 2:
            slot[2] = -1
    gates = rng.uniform(0.1, 1, size=(T, k)).astype(np.float32) if slots else None
    wide = lambda r: bf16(rng.normal(size=(r, N + pad + offset)))
    cut = lambda pair: (pair[0][:, offset:offset + N], pair[1][:, offset:offset + N])
    Y, Yv = cut(wide(rows))
    R, Rv = cut(wide(T)) if resid else (None, None)
    vec = lambda: bf16(rng.normal(size=N) + 1)
    wp, wpv = vec() if post else (None, None)
    wn, wnv = vec() if pre else (None, None)
    new = lambda: torch.full((T, N + pad + offset), 7.0, dtype=torch.bfloat16, device="cuda")
    H, Nrm = new(), new()
    ld = N + pad + offset
    if slots and skip:
        Y[~np.isin(np.arange(rows), slot)] = float("nan")   # rows nobody takes are not read into any sum
    mx.mxfp4_moe_combine(H[:, offset:] if h_out else None, ld, Nrm[:, offset:] if norm else None, ld, Y, ld, rows,
                         None if slot is None else dev(slot), None if gates is None else dev(gates), k, R, ld, wp, wn,
                         0.75, -1.5, 1e-5, T, N)
    torch.cuda.synchronize()
    s = slot if slots else np.arange(T)[:, None]
    g = gates if slots else np.ones((T, 1))
    h, n, mh, mn = ref.combine(Yv, s, g.astype(np.float64), Rv, wpv, wnv, 0.75, -1.5, 1e-5)
    for out, want, mag, on in ((H, h, mh, h_out), (Nrm, n, mn, norm)):
        got = bf16_bits_to_f64(d_to_bits(out))
        if not on:
            assert (got == 7.0).all()
            continue
        body = got[:, offset:offset + N]
        err, bound = np.abs(body - want), ulp_bf16(want) + 2.0 ** -18 * mag
        assert (err <= bound).all(), (np.argwhere(~(err <= bound))[:5], np.nanmax(err / bound))
        assert (got[:, :offset] == 7.0).all() and (got[:, offset + N:] == 7.0).all()


@pytest.mark.parametrize("T,k,N", [(1, 1, 1), (1, 8, 7168), (3, 2, 7), (5, 4, 264), (33, 3, 1000), (400, 2, 2048), (9, 16, 4104),
                                   (2, 2, 8192), (2, 1, 32768), (3, 2, 20001)])
def test_combine(T, k, N):
    check_combine(T, k, N)


def test_combine_options():
    check_combine(20, 3, 512, post=False)
    check_combine(20, 3, 512, resid=False, pre=False)
    check_combine(20, 3, 512, norm=False)
    check_combine(20, 3, 512, h_out=False, post=False)
    check_combine(20, 3, 515, pad=5, rows=90, skip=0.4)
    check_combine(20, 3, 512, offset=1, pad=7)              # rows that start off a 16-byte boundary
    check_combine(20, 1, 768, slots=False)


@pytest.mark.parametrize("T,k,N,kw", [(700, 3, 2048, {}), (615, 2, 4096, dict(skip=0.4, rows=2000)),
                                      (640, 1, 8200, dict(pad=8)), (609, 2, 2064, dict(resid=False, norm=False)),
                                      (620, 2, 2048, dict(post=False, pre=False, h_out=False)), (611, 1, 3000, dict(slots=False))])
def test_combine_many_long_rows(T, k, N, kw):
    """The form that streams rows ahead of the token at work."""
    check_combine(T, k, N, **kw)


@pytest.mark.parametrize("T,k,N,kw", [(400, 2, 515, {}), (330, 3, 1002, dict(skip=0.3)), (310, 1, 2860, {}), (305, 2, 4097, {}),
                                      (304, 1, 8191, dict(post=False)), (310, 2, 300, dict(offset=1, pad=7)),
                                      (304, 2, 32, dict(pad=1)), (2, 2, 9999, {})])
def test_combine_many_rows_off_boundaries(T, k, N, kw):
    check_combine(T, k, N, **kw)


@pytest.mark.parametrize("T,k,N,kw", [(620, 2, 2049, {}), (610, 1, 2050, dict(offset=1, pad=4, skip=0.3)), (609, 2, 4098, {}),
                                      (611, 1, 4100, dict(pad=8)), (609, 1, 8191, dict(post=False)),
                                      (608, 1, 8196, dict(resid=False)), (608, 1, 16383, dict(pre=False)),
                                      (640, 2, 2056, dict(offset=4, pad=4)), (612, 1, 2055, dict(slots=False, norm=False))])
def test_combine_many_long_rows_off_boundaries(T, k, N, kw):
    """Streamed rows that begin and end inside 16 bytes, the tensors' first and last among them."""
    check_combine(T, k, N, **kw)


@pytest.mark.parametrize("T,N", [(50, 1024), (900, 2048), (50, 1023), (700, 2049)])
def test_combine_in_place_on_the_residual(T, N):
    k = 2
    rng = np.random.default_rng(1)
    Y, Yv = bf16(rng.normal(size=(T * k, N)))
    R, Rv = bf16(rng.normal(size=(T, N)))
    slot = rng.permutation(T * k).reshape(T, k).astype(np.int32)
    gates = rng.uniform(size=(T, k)).astype(np.float32)
    mx.mxfp4_moe_combine(R, N, None, 0, Y, N, T * k, dev(slot), dev(gates), k, R, N, None, None, 1.0, 1.0, 1e-6, T, N)
    torch.cuda.synchronize()
    h, _, m, _ = ref.combine(Yv, slot, gates.astype(np.float64), Rv, None, None, 1.0, 1.0, 1e-6)
    assert (np.abs(bf16_bits_to_f64(d_to_bits(R)) - h) <= ulp_bf16(h) + 2.0 ** -18 * m).all()


# -------------------------------------------------------------------- block --


@pytest.mark.parametrize("T,E,k,K,F", [(1, 8, 3, 256, 96), (70, 6, 2, 288, 160), (0, 4, 2, 64, 64)])
def test_moe_block_runs_its_steps(T, E, k, K, F):
    """The one-call block gives what its steps give, bit for bit, and the
    router in front of it feeds both."""
    rng = np.random.default_rng(T + K)
    w1 = rng.integers(0, 256, size=(E, 2, F, K // 2), dtype=np.uint8)
    w2 = rng.integers(0, 256, size=(E, K, F // 2), dtype=np.uint8)
    s1 = rng.integers(118, 122, size=(E, 2, F, K // 32)).astype(np.uint8)
    s2 = rng.integers(118, 122, size=(E, K, F // 32)).astype(np.uint8)
    x, _ = bf16(rng.normal(size=(T, K)))
    resid, _ = bf16(rng.normal(size=(T, K)))
    logits = dev(rng.normal(size=(T, E)).astype(np.float32))
    mask = (rng.uniform(size=T) < 0.8).astype(np.uint8)
    r1, r2 = mx.relaid_expert_scales(dev(s1), K), mx.relaid_expert_scales(dev(s2), F)
    np.testing.assert_array_equal(host(r1)[E - 1, 1], ref.relaid(s1[E - 1, 1], K))
    w_pre, _ = bf16(rng.normal(size=K))
    w1, w2 = dev(w1), dev(w2)
    h, n = mx.moe_block(x, logits, resid, w1, r1, w2, r2, k, w_pre=w_pre, token_mask=dev(mask))
    torch.cuda.synchronize()
    assert h.shape == (T, K) and torch.isfinite(h.float()).all()
    if T == 0:
        return
    ids, gates, offsets, _, slot_row = run_route(logits, k, 0, dev(mask))
    Q, S = run_quantize("e2m1", x, K, slot_row, ids, offsets, E, T * k)
    p = object.__new__(Grouped)
    p.fmt = p.fmt_b = "e2m1"
    p.N, p.K, p.E, p.rows, p.lda, p.ldb = F, K, E, T * k, K, K
    p.dA, p.dSA, p.dB, p.dSB, p.dO = dev(Q), dev(S), w1, r1, dev(offsets)
    H, SH = p.swiglu()
    q = object.__new__(Grouped)
    q.fmt = q.fmt_b = "e2m1"
    q.N, q.K, q.E, q.rows, q.lda, q.ldb = K, F, E, T * k, F, F
    q.dA, q.dSA, q.dB, q.dSB, q.dO = H, SH, w2, r2, p.dO
    Y = q.gemm()
    h2, n2 = torch.empty_like(h), torch.empty_like(n)
    mx.mxfp4_moe_combine(h2, K, n2, K, Y, K, T * k, dev(slot_row), dev(gates), k, resid, K, None, w_pre, 1.0, 1.0, 1e-6, T, K)
    torch.cuda.synchronize()
    assert torch.equal(h, h2) and torch.equal(n, n2)
