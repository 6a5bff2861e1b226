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


# ------------------------------------------------------- the block as a whole --


def f64(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda().double()


def block_bounds(w, x, logits, resid, k, mask, w_pre, w_post, res_scale, out_scale, eps):
    """(h, bound of its error, n, bound of its error) from the definition, in 64 bits."""
    E, K, F = w.E, w.K, w.F
    xv = x.double().cpu().numpy()
    T = len(xv)
    ids, gates, offsets, row_token, slot_row = ref.route_many(logits.double().cpu().numpy(), k, 0, mask)
    xq = f64(ref.values(*ref.quantise(xv, "e2m1"), "e2m1"))
    Y, dY = np.zeros((T * k, K)), np.zeros((T * k, K))
    exps = np.vectorize(lambda v: ref.scale_exponent(v, "e2m1"), otypes=[int])

    def rounded(v, s):
        c, neg = ref.to_codes(np.ldexp(v, -s), "e2m1")
        return np.ldexp(ref.E2M1[c] * np.where(neg, -1, 1), s)

    for e in range(E):
        a, b = offsets[e], offsets[e + 1]
        if a == b:
            continue
        A, B1 = xq[row_token[a:b]], f64(ref.values(w.q1[e], w.c1[e], "e2m1"))
        gu, mag = (A @ B1.T).cpu().numpy(), (A.abs() @ B1.abs().T).cpu().numpy() * 2.0 ** -20
        g, u, dg, du = gu[:, :F], gu[:, F:], mag[:, :F], mag[:, F:]
        with np.errstate(over="ignore"):
            silu = g / (1 + np.exp(-g))
        h = silu * u
        d = 1.1 * np.abs(u) * dg + np.abs(silu) * du + 1.1 * dg * du + 2.0 ** -19 * (1 + np.abs(g)) * np.abs(h) + 1e-38
        spread = []
        for edge in ((np.abs(h) - d).clip(0), np.abs(h) + d):          # the scales that the block may get
            s = np.repeat(exps(edge.reshape(b - a, -1, 32).max(-1)), 32, axis=1)
            spread += [rounded(h - d, s), rounded(h + d, s)]
        low, high = np.minimum.reduce(spread), np.maximum.reduce(spread)
        assert (high - low > 0).mean() < 1e-2                           # only values beside a rounding's edge are open
        H, dH, B2 = f64((low + high) / 2), f64((high - low) / 2), f64(ref.values(w.q2[e], w.c2[e], "e2m1"))
        y = (H @ B2.T).cpu().numpy()
        err = ((dH * (1 + 2.0 ** -20) + H.abs() * 2.0 ** -20) @ B2.abs().T).cpu().numpy()
        Y[a:b], dY[a:b] = y, err + ulp_bf16(np.abs(y) + err)
    b, db, m = np.zeros((T, K)), np.zeros((T, K)), np.zeros((T, K))
    for j in range(k):
        took = slot_row[:, j] >= 0
        r, gate = slot_row[took, j], gates[took, j, None]
        b[took] += gate * Y[r]
        db[took] += gate * (dY[r] + (E / 32 + 16) * 2.0 ** -23 * (np.abs(Y[r]) + dY[r]))
        m[took] += gate * (np.abs(Y[r]) + dY[r])

    def normed(v, dv, m, weight):
        r = 1 / np.sqrt((v * v).mean(1, keepdims=True) + eps)
        q = r * np.sqrt((dv * dv).mean(1, keepdims=True))
        return v * r * weight, r * np.abs(weight) * (dv + np.abs(v) * q) / (1 - q), m * r * np.abs(weight) / (1 - q)

    if w_post is not None:
        b, db, m = normed(b, db, m, w_post.double().cpu().numpy())
    res = res_scale * resid.double().cpu().numpy()
    h, dh, m = out_scale * b + res, abs(out_scale) * db, abs(out_scale) * m + np.abs(res)
    n, dn, mn = normed(h, dh, m, 1.0 if w_pre is None else w_pre.double().cpu().numpy())
    bound = lambda v, dv, m: dv + 2.0 ** -18 * m + ulp_bf16(np.abs(v) + dv)
    return h, bound(h, dh, m), n, bound(n, dn, mn)


@pytest.mark.parametrize("T,E,k,K,F,post", [(1, 8, 3, 4096, 256, False), (300, 64, 2, 512, 192, True), (700, 6, 2, 1312, 544, False),
                                            (2048, 8, 4, 2048, 1024, False), (640, 3, 1, 1312, 2080, True)],
                         ids=["one token", "single CTAs", "pairs, streamed join", "tiles in rounds", "few experts"])
def test_block_against_the_definition(T, E, k, K, F, post):
    w = Weights(E, K, F, seed=T)
    x, logits, resid = inputs(T, E, K, seed=T + 1)
    mask = (np.random.default_rng(T).uniform(size=T) < 0.9).astype(np.uint8)
    mask[0] = 1
    g = torch.Generator(device="cuda").manual_seed(3)
    w_pre = (1 + 0.2 * torch.randn(K, device="cuda", generator=g)).bfloat16()
    w_post = (1 + 0.2 * torch.randn(K, device="cuda", generator=g)).bfloat16() if post else None
    got = w(x, logits, resid, k, w_pre=w_pre, w_post=w_post, token_mask=dev(mask), res_scale=0.75, out_scale=-0.5, eps=1e-5)
    torch.cuda.synchronize()
    h, dh, n, dn = block_bounds(w, x, logits, resid, k, mask, w_pre, w_post, 0.75, -0.5, 1e-5)
    for t, want, bound in ((got[0], h, dh), (got[1], n, dn)):
        err = np.abs(t.double().cpu().numpy() - want)
        assert (err <= bound).all(), (np.argwhere(~(err <= bound))[:5], np.nanmax(err / bound))
        assert np.median(bound / (np.abs(want) + 0.1)) < 0.05            # a bound that says something


SIZES = [(1, 8, 3, 1024, 512), (40, 16, 2, 512, 288), (700, 4, 2, 1312, 544), (1300, 4, 2, 2048, 1024)]


class InPlace:
    """Layers one after another on a residual stream that they update in place, in one workspace."""

    def __init__(self, T, E, k, K, F):
        self.size = T, E, k, K, F
        self.layers = [Weights(E, K, F, seed=s) for s in (1, 2)]
        self.x, self.logits, self.resid = inputs(T, E, K, seed=5)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.ids, self.slot_row = torch.empty((T, k), **i32), torch.empty((T, k), **i32)
        self.offsets, self.row_token = torch.empty(E + 1, **i32), torch.empty(T * k, **i32)
        self.gates = torch.empty((T, k), device="cuda")
        need = max(mx.mxfp4_moe_route_workspace_size(T, E), mx.mxfp4_moe_ffn_workspace_size(T, E, k, K, F), 256)
        self.ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def run(self, steps, between):
        T, E, k, K, F = self.size
        stream, x, outs = self.resid.clone(), self.x.clone(), []
        for i in range(steps):
            w, logits = self.layers[i % 2], self.logits.roll(i, 1)      # another routing for each step
            between(self.ws)
            mx.mxfp4_moe_route(self.ids, self.gates, self.offsets, self.row_token, self.slot_row, logits, E, mx.MXFP4_LOGITS_FP32, None,
                               T, E, k, mx.MXFP4_GATE_TOPK, 1.0, self.ws, self.ws.numel())
            mx.mxfp4_moe_ffn(stream, K, x, K, x, K, self.ids, self.gates, self.offsets, self.slot_row, T, E, k, K, F, w.w1, K, w.s1,
                             w.w2, F, w.s2, stream, K, None, None, 0.9, 0.1, 1e-6, self.ws, self.ws.numel())
            outs += [stream.clone(), x.clone()]
        torch.cuda.synchronize()
        return outs


@pytest.mark.parametrize("T,E,k,K,F", SIZES)
def test_blocks_back_to_back_on_one_workspace(T, E, k, K, F):
    """Routing and block, launch behind launch, H on top of the residual rows and the norm on top of the
    block's input, give what they give when each call has the device and a spoiled workspace to itself."""
    chain = InPlace(T, E, k, K, F)

    def alone(ws):
        torch.cuda.synchronize()
        ws.fill_(0xFF)
        torch.cuda.synchronize()

    want = chain.run(8, alone)
    assert all(torch.isfinite(t.float()).all() for t in want)
    for _ in range(4):
        assert same(chain.run(8, lambda ws: None), want)


@pytest.mark.parametrize("T,E,k,K,F", SIZES)
def test_a_block_in_a_graph_with_other_routing(T, E, k, K, F):
    w = Weights(E, K, F)
    x, logits, resid = inputs(T, E, K, seed=1)
    w(x, logits, resid, k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = [w(x, logits, resid, k) for _ in range(2)]               # two behind one another
    for seed in (2, 3, 4):
        for t, new in zip((x, logits, resid), inputs(T, E, K, seed)):
            t.copy_(new)
        if seed == 4:
            logits[:, 1:] -= 100                                       # nearly all rows with one expert
        graph.replay()
        want = w(x, logits, resid, k)
        assert same(got[0], want) and same(got[1], want)
