"""What the header says of the dense layer's operators at the far ends of their arguments."""
import pytest

import block_scaled_mxfp4_gb300 as mx
from test_gpu_dense import Product, workspace

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


# Row by row (CTA pairs, one tile a CTA), swapped operands, sums in a cluster and in the workspace of either.
PLAIN = [("mxfp4", 2560, 2304, 512, 0), ("mxfp8", 2560, 2304, 512, 0), ("mxfp8", 700, 1100, 384, 0), ("mxfp4", 1, 256, 512, 0),
         ("mxfp8", 64, 333, 4096, 0), ("mxfp4", 33, 160, 8192, 0), ("mxfp4", 7, 97, 8192, 3), ("mxfp8", 40, 64, 2048, 7),
         ("mxfp4", 9, 200, 8192, 16), ("mxfp4", 300, 500, 4096, 4), ("mxfp8", 130, 290, 2048, 5), ("mxfp8", 257, 129, 1024, 8),
         ("mxfp8", 140, 200, 4096, 11), ("mixed", 3, 2, 32, 0)]


@pytest.mark.parametrize("form,M,N,K,split", PLAIN)
def test_product_without_epilogue_has_the_gemms_zeros(form, M, N, K, split):
    """The same bits as the plain product, the signs of zeros among them: sums that are 0 and
    products with alpha that underflow, of either sign."""
    p = Product(form, M, N, K, 11)
    p.dA[M // 2] = 0
    p.dB[:: max(1, N // 3)] = 0
    size = mx.mxfp4_gemm_workspace_size if form == "mxfp4" else mx.mxfp8_gemm_workspace_size
    ws = workspace(size(M, N, K, split))
    for alpha in (-p.alpha, p.alpha, -2.0 ** -149, 2.0 ** -149):
        got = p.run(split_k=split, alpha=alpha)[0]
        want = torch.empty_like(got)
        args = (want, N, None, 0, p.dA, K, p.dB, K, p.dSA, K // 32, p.dSB, K // 32)
        if form == "mxfp4":
            mx.mxfp4_gemm(*args, alpha, 0.0, M, N, K, split, ws, ws.numel())
        else:
            mx.mxfp8_gemm(*args, *p.fmts, alpha, 0.0, M, N, K, split, ws, ws.numel())
        torch.cuda.synchronize()
        assert (want == 0).any()
        assert torch.equal(got.view(torch.int16), want.view(torch.int16)), alpha
