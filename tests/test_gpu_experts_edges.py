"""Expert-layer operators where indexes pass 32 bits and where masked places hold
what must not come through.  The big arrays are strides, not work: 9 to 13 GB, of
which a few rows are touched."""
import numpy as np
import pytest

import block_scaled_mxfp4_gb300 as mx
import expert_ref as ref
from parity_util import bf16_bits_to_f64, d_to_bits, ulp_bf16
from test_gpu_experts import Grouped, host, run_route

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


@pytest.fixture(autouse=True)
def _memory():
    yield
    torch.cuda.empty_cache()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def apart(t, ld):
    """The same rows, ld elements from one to the next."""
    wide = torch.empty(((t.shape[0] - 1) * ld + t.shape[1],), dtype=t.dtype, device="cuda")
    out = wide.as_strided(t.shape, (ld, 1))
    out.copy_(t)
    return out


FAR = 1 << 27                                              # 34 such rows pass 2^32 bytes and elements


@pytest.mark.parametrize("counts", [[3, 0, 25], [20, 14], [0, 34]], ids=["32 rows", "single CTAs", "one group"])
@pytest.mark.parametrize("N", [96, 101])
def test_products_with_rows_far_apart(counts, N):
    p = Grouped(counts, N, 160, seed=1)
    want = host(p.gemm().view(torch.int16))
    A = apart(p.dA, FAR // 2)
    D = apart(torch.full((p.rows, N), 7.0, dtype=torch.bfloat16, device="cuda"), FAR + (N & 1))
    mx.mxfp4_grouped_gemm(D, FAR + (N & 1), A, FAR, p.dSA, p.dB, p.ldb, N * p.ldb, p.dSB, p.dO, p.E, p.rows, N, p.K, 1.0, None, 0)
    np.testing.assert_array_equal(host(D.contiguous().view(torch.int16)), want)


def test_pairs_with_rows_far_apart():
    p = Grouped([300, 290], 264, 160, seed=1)
    want = host(p.gemm().view(torch.int16))
    ld = 1 << 23                                           # 590 rows
    A, D = apart(p.dA, ld // 2), apart(torch.full((p.rows, p.N), 7.0, dtype=torch.bfloat16, device="cuda"), ld)
    mx.mxfp4_grouped_gemm(D, ld, A, ld, p.dSA, p.dB, p.ldb, p.N * p.ldb, p.dSB, p.dO, p.E, p.rows, p.N, p.K, 1.0, None, 0)
    np.testing.assert_array_equal(host(D.contiguous().view(torch.int16)), want)


@pytest.mark.parametrize("counts,ld", [([3, 0, 25], 1 << 28), ([300, 290], 1 << 24)])
def test_gated_rows_and_weights_far_apart(counts, ld):
    p = Grouped(counts, 96, 160, halves=2, seed=1)
    want = [host(t) for t in p.swiglu(alpha=0.01)]
    H = apart(torch.full((p.rows, 48), 0xEE, dtype=torch.uint8, device="cuda"), ld // 2)
    S = torch.full((mx.mxfp4_group_scale_size(p.rows, p.E, 96),), 0xDD, dtype=torch.uint8, device="cuda")
    far = 1 << 33                                          # elements between two experts' weights
    B = apart(p.dB.reshape(p.E, -1), far // 2)
    mx.mxfp4_grouped_swiglu(H, ld, S, p.dA, p.lda, p.dSA, B, p.ldb, far, p.dSB, p.dO, p.E, p.rows, 96, p.K, 0.01, None, 0)
    np.testing.assert_array_equal(host(H.contiguous()), want[0])
    np.testing.assert_array_equal(host(S), want[1])


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_quantiser_with_rows_far_apart(fmt):
    T, E, k, K = 20, 5, 2, 288
    rng = np.random.default_rng(1)
    ids = np.argsort(rng.uniform(size=(T, E)), axis=1)[:, :k].astype(np.int32)
    offsets, row_token, slot_row = ref.grouping(ids, E)
    x = dev(rng.normal(size=(T, K))).to(torch.bfloat16)
    width = K // 2 if fmt == "e2m1" else K
    Q = apart(torch.full((T * k, width), 0xEE, dtype=torch.uint8, device="cuda"), FAR)
    S = torch.full((mx.mxfp4_group_scale_size(T * k, E, K),), 0xDD, dtype=torch.uint8, device="cuda")
    far = apart(x, FAR)
    args = (S, far, FAR, T, K, dev(slot_row), dev(ids), k, dev(offsets), E, T * k)
    if fmt == "e2m1":
        mx.mxfp4_group_quantize(Q, 2 * FAR, *args)
    else:
        mx.mxfp8_group_quantize(Q, FAR, *args, mx.MXFP8_E4M3)
    codes, scales = ref.quantise(x.double().cpu().numpy(), fmt)
    np.testing.assert_array_equal(host(Q.contiguous()), codes[row_token])
    np.testing.assert_array_equal(host(S)[ref.scale_places(offsets, K)], scales[row_token])


@pytest.mark.parametrize("T,E", [(20, 40), (100, 300)])
def test_router_with_rows_far_apart(T, E):
    x = torch.randn((T, E), device="cuda")
    far = apart(x, (1 << 33) // 4 // T + 5)
    for kind in (0, 1):
        got, want = run_route(far, 3, kind), run_route(x, 3, kind)
        for a, b in zip(got, want):
            np.testing.assert_array_equal(a, b)


@pytest.mark.parametrize("T,N,far", [(9, 264, FAR), (9, 265, FAR), (620, 1288, 1 << 22), (620, 1301, (1 << 22) + 1)],
                         ids=["few", "few, off boundaries", "streamed", "streamed, off boundaries"])
def test_join_with_rows_far_apart(T, N, far):
    """Rows of Y past 2^32 elements, residual and results too."""
    rng = np.random.default_rng(N)
    k, rows = 2, max(34, 2 * T)
    Y, R = (dev(rng.normal(size=(n, N))).to(torch.bfloat16) for n in (rows, T))
    slots = rng.permutation(rows)[:T * k].reshape(T, k).astype(np.int32)
    slots[0, 0] = rows - 1
    slots[1, 1] = -1
    gates = torch.rand((T, k), device="cuda")
    h, n = (torch.empty((T, N), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    mx.mxfp4_moe_combine(h, N, n, N, Y, N, rows, dev(slots), gates, k, R, N, None, None, 1.0, 1.0, 1e-6, T, N)
    wideY, wide = apart(Y, far), [apart(t, far) for t in (R, torch.zeros_like(h), torch.zeros_like(n))]
    mx.mxfp4_moe_combine(wide[1], far, wide[2], far, wideY, far, rows, dev(slots), gates, k, wide[0], far, None, None, 1.0, 1.0,
                         1e-6, T, N)
    torch.cuda.synchronize()
    assert torch.equal(wide[1], h) and torch.equal(wide[2], n)


@pytest.mark.parametrize("T,N", [(40, 512), (40, 515), (700, 2048), (700, 2049)])
def test_join_takes_nothing_from_masked_places(T, N):
    """Gates and rows of slots that are not taken hold NaN and infinities."""
    rng = np.random.default_rng(N)
    k, rows = 4, 5 * T
    slots = rng.permutation(rows)[:T * k].reshape(T, k).astype(np.int32)
    slots[rng.uniform(size=slots.shape) < 0.4] = -1
    slots[3] = -1
    slots[4, 1:] = -1
    slots[5, 0] = rows + 3                                 # a row that cannot be
    gates = rng.uniform(size=(T, k)).astype(np.float32)
    taken = (slots >= 0) & (slots < rows)
    Yv = rng.normal(size=(rows, N))
    Y, R = dev(Yv).to(torch.bfloat16), dev(rng.normal(size=(T, N))).to(torch.bfloat16)
    Yv = Y.double().cpu().numpy()
    Y[dev(~np.isin(np.arange(rows), slots[taken]))] = float("nan")
    spoiled = np.where(taken, gates, rng.choice([np.nan, np.inf, -np.inf], size=gates.shape)).astype(np.float32)
    h, n = (torch.empty((T, N), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    mx.mxfp4_moe_combine(h, N, n, N, Y, N, rows, dev(slots), dev(spoiled), k, R, N, None, None, 1.0, 1.0, 1e-6, T, N)
    torch.cuda.synchronize()
    Rv = R.double().cpu().numpy()
    wh, wn, mh, mn = ref.combine(Yv, np.where(taken, slots, -1), gates.astype(np.float64), Rv, None, None, 1.0, 1.0, 1e-6)
    for got, want, mag in ((h, wh, mh), (n, wn, mn)):
        assert (np.abs(bf16_bits_to_f64(d_to_bits(got)) - want) <= ulp_bf16(want) + 2.0 ** -18 * mag).all()


@pytest.mark.parametrize("T", [1, 30, 700])
def test_block_takes_nothing_from_masked_tokens(T):
    """Tokens without experts hold NaN in the block's input and in their logits."""
    E, k, K, F = 5, 2, 1312, 96
    rng = np.random.default_rng(T)
    u8 = lambda lo, hi, *shape: dev(rng.integers(lo, hi, size=shape).astype(np.uint8))
    w1, w2 = u8(0, 256, E, 2, F, K // 2), u8(0, 256, E, K, F // 2)
    s1 = mx.relaid_expert_scales(u8(118, 122, E, 2, F, K // 32), K)
    s2 = mx.relaid_expert_scales(u8(118, 122, E, K, F // 32), F)
    x, resid = (dev(rng.normal(size=(T, K))).to(torch.bfloat16) for _ in range(2))
    logits = dev(rng.normal(size=(T, E)).astype(np.float32))
    mask = dev(rng.uniform(size=T) < 0.5)
    mask[0] = False
    want = mx.moe_block(x, logits, resid, w1, s1, w2, s2, k, token_mask=mask)
    x[~mask], logits[~mask] = float("nan"), float("inf")
    got = mx.moe_block(x, logits, resid, w1, s1, w2, s2, k, token_mask=mask)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.isfinite(got[0].float()).all()
    assert torch.equal(got[0][~mask], resid[~mask])
