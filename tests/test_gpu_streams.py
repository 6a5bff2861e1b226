"""The entries that allocate for their caller, on another stream than the
current one: what they allocate, copy and drop has to belong to that stream.
The stream is kept busy while the current one allocates and overwrites memory
of every size that the entry used, so that memory handed out too early shows."""
import numpy as np
import pytest

import block_scaled_mxfp4_gb300 as mx
import expert_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from block_scaled_mxfp4_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def busy(stream):
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        torch.cuda._sleep(40_000_000)                      # some 20 ms


def churn(sizes):
    """Memory of these sizes, allocated and overwritten on the current stream."""
    held = [torch.full((n,), 0x77, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
    torch.cuda.current_stream().synchronize()              # overwritten while the other stream still sleeps
    return held


@pytest.mark.parametrize("as_handle", [False, True])
@pytest.mark.parametrize("T", [5, 200])
def test_moe_block_on_another_stream(T, as_handle):
    E, k, K, F = 6, 2, 256, 96
    rng = np.random.default_rng(T)
    w1 = dev(rng.integers(0, 256, size=(E, 2, F, K // 2), dtype=np.uint8))
    w2 = dev(rng.integers(0, 256, size=(E, K, F // 2), dtype=np.uint8))
    r1 = mx.relaid_expert_scales(dev(rng.integers(118, 122, size=(E, 2, F, K // 32)).astype(np.uint8)), K)
    r2 = mx.relaid_expert_scales(dev(rng.integers(118, 122, size=(E, K, F // 32)).astype(np.uint8)), F)
    x, resid = (dev(rng.normal(size=(T, K))).to(torch.bfloat16) for _ in range(2))
    logits = dev(rng.normal(size=(T, E)).astype(np.float32))
    h0, n0 = mx.moe_block(x, logits, resid, w1, r1, w2, r2, k)
    side = torch.cuda.Stream()
    ws = max(mx.mxfp4_moe_route_workspace_size(T, E), mx.mxfp4_moe_ffn_workspace_size(T, E, k, K, F), 256)
    for _ in range(3):
        busy(side)
        h, n = mx.moe_block(x, logits, resid, w1, r1, w2, r2, k, stream=side.cuda_stream if as_handle else side)
        held = churn([T * k * 4, (E + 1) * 4, T * K * 2, ws])
        torch.cuda.synchronize()
        assert torch.equal(h, h0) and torch.equal(n, n0)
        del held


def test_relaid_expert_scales_on_another_stream():
    E, rows, K = 5, 200, 1024
    wide = dev(np.random.default_rng(2).integers(0, 255, size=(E, rows, K // 16)).astype(np.uint8))
    S = wide[:, :, ::2]                                    # the rows have to be copied first
    side = torch.cuda.Stream()
    busy(side)
    out = mx.relaid_expert_scales(S, K, stream=side)
    held = churn([E * rows * K // 32, out.numel()])
    torch.cuda.synchronize()
    for e in range(E):
        np.testing.assert_array_equal(out[e].cpu().numpy(), ref.relaid(S[e].cpu().numpy(), K))
    del held


@pytest.mark.parametrize("M,N,K,split", [(8, 512, 4096, 4), (300, 512, 1024, 0)])
def test_gemm_on_another_stream(M, N, K, split):
    g = torch.Generator(device="cuda").manual_seed(M)
    byte = lambda lo, hi, *shape: torch.randint(lo, hi, shape, dtype=torch.uint8, device="cuda", generator=g)
    A, B = byte(0, 256, M, K // 2), byte(0, 256, N, K // 2)
    SA, SB = byte(118, 122, M, K // 32), byte(118, 122, N, K // 32)
    need = mx.mxfp4_gemm_workspace_size(M, N, K, split)
    want = mx.gemm(A, B, SA, SB, split_k=split)
    side = torch.cuda.Stream()
    for _ in range(3):
        busy(side)
        got = mx.gemm(A, B, SA, SB, split_k=split, stream=side)
        held = churn([M * N * 2, max(need, 256)])
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        del held
