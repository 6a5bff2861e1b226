"""Calls of the dense layer's operators that their documentation allows beside the ordinary ones:
every byte format under the epilogue, parameters off 16-byte boundaries, few rows, two streams at
once, replays beside eager calls, and a wait limit shorter than the work ahead."""
import numpy as np
import pytest

import block_scaled_mxfp4_gb300 as mx
import dense_ref as dr
from block_scaled_mxfp4_gb300 import inputs
from test_gpu_dense import KIND, Product, bf16, check_norm, check_norm_backward, checkpoint_of, dev, host, run_backward, run_checkpoint, workspace

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BYTES = {"e4m3": mx.MXFP8_E4M3, "e5m2": mx.MXFP8_E5M2, "e2m3": mx.MXFP6_E2M3, "e3m2": mx.MXFP6_E3M2, "e2m1": mx.MXFP4_E2M1_PADDED}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from block_scaled_mxfp4_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    mx.mxfp4_device_status(reset=True)
    yield
    assert mx.mxfp4_device_status() == 0, "a bounded wait timed out during the tests"


@pytest.mark.parametrize("fa,fb", [("e2m3", "e2m3"), ("e3m2", "e4m3"), ("e4m3", "e2m1"), ("e2m1", "e5m2"), ("e5m2", "e3m2")])
@pytest.mark.parametrize("M,N,K", [(2560, 2304, 256), (2307, 2410, 160), (300, 96, 160), (3, 64, 2048)])
def test_every_byte_format_under_the_epilogue(fa, fb, M, N, K):
    """D without bias, activation and residual has the plain product's bits; with ReLU it is D's maximum with 0."""
    p = inputs.make_problem8("formats", M, N, K, M + K, fa, fb, "normal", 1.0, 0.0, None)
    A, B, SA, SB = (dev(t) for t in (p.A, p.B, p.SA, p.SB))
    need = mx.mxfp8_gemm_workspace_size(M, N, K, 0)
    ws = workspace(need)
    want, got, relu = (torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    mx.mxfp8_gemm(want, N, None, 0, A, K, B, K, SA, K // 32, SB, K // 32, BYTES[fa], BYTES[fb], 0.5, 0.0, M, N, K, 0, ws, need)
    for D, act in ((got, mx.MXFP4_ACT_NONE), (relu, mx.MXFP4_ACT_RELU)):
        mx.mxfp8_gemm_act(D, N, None, 0, None, 0, None, 0, None, 0, A, K, B, K, SA, K // 32, SB, K // 32, BYTES[fa], BYTES[fb], 0, 0, 0.5,
                          None, 0, act, None, 0, 0.0, M, N, K, 0, 0, ws, need)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(relu, want.clamp(min=0))


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("form,M,N,K", [("mxfp8", 2560, 2304, 512), ("mxfp8", 300, 96, 160), ("mxfp4", 3, 97, 8192), ("mxfp4", 130, 290, 2048)])
def test_bias_off_its_boundary(form, M, N, K, kind):
    p = Product(form, M, N, K, 3)
    t = torch.randn(N + 1, device="cuda").to(torch.bfloat16 if kind == "bf16" else torch.float32)
    a = p.run("gelu", t[1:].clone(), kind)[0]
    b = p.run("gelu", t[1:], kind)[0]
    torch.cuda.synchronize()
    assert torch.equal(a, b)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("T,N", [(7, 1000), (3000, 1024), (40, 4096), (700, 9000)])
def test_norm_parameters_off_their_boundaries(T, N, kind):
    x, dy = (torch.randn((T, N), device="cuda").bfloat16() for _ in range(2))
    w, b = (torch.randn(N + 1, device="cuda").to(torch.bfloat16 if kind == "bf16" else torch.float32) for _ in range(2))
    ws = workspace(mx.mxfp4_layer_norm_workspace_size(T, N))
    outs = []
    for w_, b_ in ((w[1:], b[1:]), (w[1:].clone(), b[1:].clone())):
        y, dx = torch.empty_like(x), torch.empty_like(x)
        m, r, dw, db = (torch.empty(n, device="cuda") for n in (T, T, N, N))
        mx.mxfp4_layer_norm(y, N, m, r, x, N, w_, b_, KIND[kind], 1e-5, T, N)
        mx.mxfp4_layer_norm_backward(dx, N, dw, db, dy, N, x, N, m, r, w_, KIND[kind], None, 0, T, N, ws, ws.numel())
        outs.append([t.double().cpu().numpy() for t in (y, dx, m, r, dw, db)])
    torch.cuda.synchronize()
    xs, dys, wv, bv = (t.double().cpu().numpy() for t in (x, dy, w[1:], b[1:]))
    v, mean, rstd, e, em, er = dr.norm(xs, wv, bv, 1e-5)
    for y, dx, m, r, dw, db in outs:
        dr.check_bf16(y, v, e, "y")
        assert (np.abs(m - mean) <= em).all() and (np.abs(r - rstd) <= er).all()
        gx, gw, gb, ex, ew, eb = dr.norm_backward(xs, dys, m, r, wv, 0.0)
        dr.check_bf16(dx, gx, ex, "dx")
        assert (np.abs(dw - gw) <= ew + 2.0 ** -140).all() and (np.abs(db - gb) <= eb + 2.0 ** -140).all()


@pytest.mark.parametrize("T,N", [(1, 1001), (2, 257), (76, 1024), (77, 1024), (75, 264), (304, 1001), (305, 999), (1215, 602), (1217, 602), (300, 1022)])
def test_norm_gradients_of_few_rows(T, N):
    for params in ((True, True), (True, False), (False, True)):
        check_norm_backward(T, N, "fp32", params=params, resid=params[0])


def test_two_streams_at_once():
    """The same inputs, workspaces of their own."""
    p = Product("mxfp8", 64, 333, 4096, 5)
    x, _ = bf16(np.random.default_rng(0).normal(size=(3000, 1024)))
    z, sz, _ = checkpoint_of(np.random.default_rng(1).normal(size=(700, 512)), "e4m3")
    dh, _ = bf16(np.random.default_rng(2).normal(size=(700, 512)))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()

    def calls(stream):
        out = []
        with torch.cuda.stream(stream):
            for _ in range(4):
                out.append([t for t in p.run("gelu", z="e4m3") if t is not None] + [t for t in run_checkpoint(x, 1024, "e4m3")] +
                           [t for t in run_backward(dh, z, sz, "e4m3", "gelu", 512)])
        return out

    both = [calls(s) for s in streams]
    torch.cuda.synchronize()
    first = both[0][0]
    for out in both:
        for one in out:
            assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(one, first))


def test_the_same_array_twice():
    """Both operands of a product, a norm's gradient and its residual, weight and bias: one array each."""
    p = Product("mxfp8", 320, 320, 512, 7)
    p.dB, p.dSB, p.B = p.dA, p.dSA, p.A
    p.fmts[1] = p.fmts[0]
    p.acc, p.mag = p.A @ p.A.T, np.abs(p.A) @ np.abs(p.A).T
    p.check("silu", bias=True, z="e4m3", h="e4m3")
    T, N = 90, 640
    x, dy = (torch.randn((T, N), device="cuda").bfloat16() for _ in range(2))
    w = torch.randn(N, device="cuda")
    y, dx, m, r = torch.empty_like(x), torch.empty_like(x), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    mx.mxfp4_layer_norm(y, N, m, r, x, N, w, w, mx.MXFP4_PARAM_FP32, 1e-5, T, N)
    mx.mxfp4_layer_norm_backward(dx, N, None, None, dy, N, x, N, m, r, w, mx.MXFP4_PARAM_FP32, dy, N, T, N, None, 0)
    xs, ws = host(x), host(w)
    v, _, _, e, _, _ = dr.norm(xs, ws, ws, 1e-5)
    dr.check_bf16(host(y), v, e, "y")
    gx, _, _, ex, _, _ = dr.norm_backward(xs, host(dy), host(m), host(r), ws, host(dy))
    dr.check_bf16(host(dx), gx, ex, "dx")


def test_a_wait_limit_shorter_than_the_work_ahead():
    """The limit counts a kernel's own waits: each of these starts while a long one runs, as its
    programmatic dependent, and waits for that without a limit."""
    rows, cols = 16384, 16384                             # some 450 us, 800,000 cycles
    dh = torch.randn((rows, cols), device="cuda").bfloat16()
    z = torch.randint(0, 120, (rows, cols), dtype=torch.uint8, device="cuda")
    sz = torch.full((rows, cols // 32), 125, dtype=torch.uint8, device="cuda")
    qt, st = torch.empty((cols, rows), dtype=torch.uint8, device="cuda"), torch.empty((cols, rows // 32), dtype=torch.uint8, device="cuda")

    def long():
        mx.mxfp8_act_backward(None, 0, None, 0, None, 0, qt, rows, st, rows // 32, None, 0, None, 0, None, dh, cols, z, cols, sz, cols // 32,
                              0, mx.MXFP4_ACT_GELU, rows, cols, 0, 0, None, 0)

    T, N = 3000, 1024
    x, _ = bf16(np.random.default_rng(0).normal(size=(T, N)))
    zz, szz, _ = checkpoint_of(np.random.default_rng(1).normal(size=(T, N)), "e4m3")
    m, r, dw, db = (torch.empty(n, device="cuda") for n in (T, T, N, N))
    y, dx = torch.empty_like(x), torch.empty_like(x)
    ws = workspace(mx.mxfp4_layer_norm_workspace_size(T, N))
    steps = [lambda: mx.mxfp4_layer_norm(y, N, m, r, x, N, None, None, 0, 1e-5, T, N),
             lambda: mx.mxfp4_layer_norm_backward(dx, N, dw, db, x, N, x, N, m, r, None, 0, x, N, T, N, ws, ws.numel()),
             lambda: run_checkpoint(x, N, "e4m3"), lambda: run_backward(x, zz, szz, "e4m3", "silu", N)]
    for step in steps:
        step()
    torch.cuda.synchronize()
    mx.mxfp4_device_status(reset=True)
    mx.mxfp4_set_wait_limit(400_000)
    try:
        for step in steps:
            long()
            step()
        torch.cuda.synchronize()
        assert mx.mxfp4_device_status() == 0
    finally:
        mx.mxfp4_set_wait_limit(1 << 32)


def test_replays_beside_eager_calls_of_the_same_leaves():
    """A captured backward pass replayed while an eager one of the same arrays is in flight on another stream."""
    T, N = 500, 512
    x, _ = bf16(np.random.default_rng(3).normal(size=(T, N)))
    z, sz, _ = checkpoint_of(np.random.default_rng(4).normal(size=(T, N)), "e4m3")
    want = [t.clone() for t in run_backward(x, z, sz, "e4m3", "gelu", N) if t is not None]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = run_backward(x, z, sz, "e4m3", "gelu", N)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(s):
            eager = run_backward(x, z, sz, "e4m3", "gelu", N)
        g.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, [t for t in captured if t is not None], [t for t in eager if t is not None]):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)) and torch.equal(a.view(torch.uint8), c.view(torch.uint8))


@pytest.mark.parametrize("T,N", [(90, 640), (5, 640), (500, 200), (3000, 1024), (400, 2000), (700, 9000), (400, 17000)])
def test_norm_gradient_without_sums_or_workspace(T, N):
    x, dy = (torch.randn((T, N), device="cuda").bfloat16() for _ in range(2))
    m, r = x.float().mean(1), torch.ones(T, device="cuda")
    want, got = torch.empty_like(x), torch.empty_like(x)
    ws = workspace(mx.mxfp4_layer_norm_workspace_size(T, N))
    dw = torch.empty(N, device="cuda")
    mx.mxfp4_layer_norm_backward(want, N, dw, dw.clone(), dy, N, x, N, m, r, None, 0, None, 0, T, N, ws, ws.numel())
    mx.mxfp4_layer_norm_backward(got, N, None, None, dy, N, x, N, m, r, None, 0, None, 0, T, N, None, 0)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("form,M,N,K", [("mxfp8", 2560, 2304, 512), ("mxfp8", 300, 96, 160), ("mxfp4", 3, 97, 8192), ("mxfp4", 130, 290, 2048)])
@pytest.mark.parametrize("act", dr.ACTS)
def test_infinite_and_missing_biases_stay_in_their_columns(form, M, N, K, act):
    p = Product(form, M, N, K, 4)
    bias = torch.randn(N, device="cuda")
    want = p.run(act, bias, "fp32")[0]
    odd = bias.clone()
    odd[1], odd[40], odd[65] = float("inf"), float("-inf"), float("nan")
    got = p.run(act, odd, "fp32")[0]
    torch.cuda.synchronize()
    assert (got[:, 1] == float("inf")).all() and got[:, 65].isnan().all()
    low = got[:, 40]
    assert {"none": low == float("-inf"), "relu": low == 0, "gelu": low == 0}.get(act, low.isnan()).all()
    keep = torch.ones(N, dtype=torch.bool, device="cuda")
    keep[[1, 40, 65]] = False
    assert torch.equal(got[:, keep], want[:, keep])


@pytest.mark.parametrize("T,N", [(305, 6001), (305, 8191), (460, 1501), (609, 3001), (913, 301), (1217, 701), (1300, 258), (39, 8191), (38, 8192), (77, 4097),
                                 (76, 4104), (97, 4096), (263, 1500), (300, 1501), (192, 2048), (193, 2048), (200, 1030)])
def test_norms_between_few_and_many_rows(T, N):
    check_norm(T, N, "fp32")
    check_norm_backward(T, N, "bf16")
    need = mx.mxfp4_layer_norm_workspace_size(T, N)          # nothing behind the workspace is written
    ws = workspace(need + (1 << 20))
    x, dy = (torch.randn((T, N), device="cuda").bfloat16() for _ in range(2))
    m, r = torch.zeros(T, device="cuda"), torch.ones(T, device="cuda")
    dx, dw, db = torch.empty_like(x), torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    mx.mxfp4_layer_norm_backward(dx, N, dw, db, dy, N, x, N, m, r, None, 0, None, 0, T, N, ws, need)
    torch.cuda.synchronize()
    assert (ws[need:] == 0xAB).all()
