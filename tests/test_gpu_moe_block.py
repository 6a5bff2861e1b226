"""The routed block as a whole: its arguments' layouts, its overlapped steps at
prefill sizes against a plain 64-bit form, calls back to back.

Bound of the plain form, from the arithmetic: with d the gated product's error
(as for mxfp4_grouped_swiglu), H's dequantised values lie between the roundings
of h - d and h + d, under any scale that an amax of that block within d allows;
that spread, through |B2|, the down product's accumulation (2^-20 sum |a b|) and
its bf16 rounding bound the rows of Y; the gates (a relative
(E / 32 + 16) 2^-23) and the join (2^-18 of its terms, one rounding) follow, and
a change e of the residual row moves its root mean square by rms(e) at most.
"""
import numpy as np
import pytest

import block_scaled_mxfp4_gb300 as mx
import expert_ref as ref
from test_gpu_experts import Grouped
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


class Weights:
    def __init__(self, E, K, F, seed=0):
        rng = np.random.default_rng(seed)
        self.E, self.K, self.F = E, K, F
        self.q1 = rng.integers(0, 256, size=(E, 2 * F, K // 2), dtype=np.uint8)
        self.q2 = rng.integers(0, 256, size=(E, K, F // 2), dtype=np.uint8)
        # Products of a few units, so that the activation sees all of its range.
        at = 127 - int(round(np.log2(2.9 * np.sqrt(K))))
        self.c1 = rng.integers(at, at + 2, size=(E, 2 * F, K // 32)).astype(np.uint8)
        self.c2 = rng.integers(at, at + 2, size=(E, K, F // 32)).astype(np.uint8)
        self.w1, self.w2 = dev(self.q1.reshape(E, 2, F, K // 2)), dev(self.q2)
        self.s1 = mx.relaid_expert_scales(dev(self.c1.reshape(E, 2, F, K // 32)), K)
        self.s2 = mx.relaid_expert_scales(dev(self.c2), F)

    def __call__(self, x, logits, resid, k, **kw):
        return mx.moe_block(x, logits, resid, self.w1, self.s1, self.w2, self.s2, k, **kw)


def inputs(T, E, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *shape: torch.randn(shape, device="cuda", generator=g)
    return rand(T, K).bfloat16(), rand(T, E), rand(T, K).bfloat16()


def same(got, want):
    torch.cuda.synchronize()
    return all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("T", [1, 37])
def test_rows_apart_and_masks_of_truth_values(T):
    w = Weights(4, 256, 96)
    x, logits, resid = inputs(T, 4, 256, T)
    mask = torch.arange(T, device="cuda") % 5 != 3
    want = w(x, logits, resid, 2, token_mask=mask.to(torch.uint8))
    wide = lambda t, n: torch.cat((t, torch.full((T, n), float("nan"), dtype=t.dtype, device="cuda")), 1)[:, :t.shape[1]]
    assert same(w(wide(x, 24), wide(logits, 3), wide(resid, 5), 2, token_mask=mask), want)
    if T == 1:                                             # a lone row's stride says nothing
        lone = lambda t: t.reshape(-1)[:, None].t()
        assert lone(x).stride(0) == 1
        assert same(w(lone(x), lone(logits), lone(resid), 2, token_mask=mask), want)


def test_logits_of_other_types_are_refused():
    w = Weights(4, 256, 96)
    x, logits, resid = inputs(9, 4, 256, 9)
    for bad in (logits.half(), logits.double()):
        with pytest.raises(TypeError):
            w(x, bad, resid, 2)


@pytest.mark.parametrize("T,N", [(5, 512), (5, 515), (700, 2048), (700, 2049)])
def test_a_join_without_rows(T, N):
    """No token has an expert and there is no row: the residual stream and its norm, in every form."""
    rng = np.random.default_rng(N)
    resid = dev(rng.normal(size=(T, N))).to(torch.bfloat16)
    Y = torch.empty((0, N), dtype=torch.bfloat16, device="cuda")
    slots, gates = torch.full((T, 2), -1, dtype=torch.int32, device="cuda"), torch.ones((T, 2), device="cuda")
    h, n = torch.empty_like(resid), torch.empty_like(resid)
    mx.mxfp4_moe_combine(h, N, n, N, Y, N, 0, slots, gates, 2, resid, N, None, None, 1.0, 1.0, 1e-6, T, N)
    torch.cuda.synchronize()
    assert torch.equal(h, resid)
    v = resid.double().cpu().numpy()
    want = v / np.sqrt((v * v).mean(1, keepdims=True) + 1e-6)
    assert (np.abs(bf16_bits_to_f64(d_to_bits(n)) - want) <= ulp_bf16(want) + 2.0 ** -18 * np.abs(want)).all()


@pytest.mark.parametrize("counts", [[10, 10, 10], [40, 0, 60, 20], [300, 250], [3] * 120 + [400]],
                         ids=["32 rows", "single CTAs", "pairs", "many groups"])
@pytest.mark.parametrize("gated", [False, True])
def test_offsets_out_of_order_write_nothing_outside(counts, gated):
    """Unordered or oversized offsets: values are unspecified, but the arrays' neighbours stay."""
    p = Grouped(counts, 320, 96, halves=2 if gated else 1)
    rows, E = p.rows, p.E
    rng = np.random.default_rng(rows)
    some = [np.arange(E + 1)[::-1] * rows // E, np.where(np.arange(E + 1) % 2, rows, 0), np.where(np.arange(E + 1) % 2, 0, rows),
            rng.integers(-rows, 3 * rows, size=E + 1), np.full(E + 1, -(1 << 31)), np.full(E + 1, (1 << 31) - 1),
            np.where(np.arange(E + 1) % 2, (1 << 31) - 1, -(1 << 31)), rng.permutation(p.offsets)]
    pad = 4096

    def guarded(n):
        t = torch.full((n + 2 * pad,), 0xAB, dtype=torch.uint8, device="cuda")
        return t, t[pad:pad + n]

    for offsets in some:
        p.dO = dev(offsets.astype(np.int32))
        if gated:
            (all_h, H), (all_s, S) = guarded(rows * p.N // 2), guarded(mx.mxfp4_group_scale_size(rows, E, p.N))
            mx.mxfp4_grouped_swiglu(H, p.N, S, p.dA, p.lda, p.dSA, p.dB, p.ldb, 2 * p.N * p.ldb, p.dSB, p.dO, E, rows, p.N, p.K, 1.0, None, 0)
            arrays = (all_h, all_s)
        else:
            all_d, D = guarded(rows * p.N * 2)
            mx.mxfp4_grouped_gemm(D, p.N, p.dA, p.lda, p.dSA, p.dB, p.ldb, p.N * p.ldb, p.dSB, p.dO, E, rows, p.N, p.K, 1.0, None, 0)
            arrays = (all_d,)
        torch.cuda.synchronize()
        assert mx.mxfp4_device_status() == 0
        for t in arrays:
            assert (t[:pad] == 0xAB).all() and (t[-pad:] == 0xAB).all()
