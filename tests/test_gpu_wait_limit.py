"""The limit on in-kernel waits counts a kernel's own work, not the work ahead
of it on the stream: a product that starts early (inside mxfp4_moe_ffn) and is
kept waiting for its rows ten times longer than the limit still gives its result."""
import ctypes
import subprocess

import numpy as np
import pytest

import block_scaled_mxfp4_gb300 as mx
from block_scaled_mxfp4_gb300 import build as mxbuild
from test_gpu_experts import Grouped, host

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

LIMIT = 400_000                     # cycles, some 0.2 ms; the products below take some 20 us
HOLD = 10 * LIMIT


@pytest.fixture(scope="module")
def early(tmp_path_factory):
    mxbuild.build()
    so = str(tmp_path_factory.mktemp("early") / "early_product.so")
    src = __file__.replace("test_gpu_wait_limit.py", "early_product.cu")
    subprocess.check_call([mxbuild.nvcc(), *mxbuild.ARCH, *mxbuild.NVCC_FLAGS, "-shared", "-o", so, src, mx.library_path(),
                           "-cudart", "static"])
    mx.lib()
    call = ctypes.CDLL(so).early_product
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    call.argtypes = [vp, i64, vp, vp, i64, vp, vp, i64, i64, vp, vp, i32, i32, i32, i32, i32, ctypes.c_longlong, vp]
    return call


@pytest.fixture
def limit():
    mx.mxfp4_device_status(reset=True)
    mx.mxfp4_set_wait_limit(LIMIT)
    yield
    mx.mxfp4_set_wait_limit(1 << 32)
    torch.cuda.synchronize()
    mx.mxfp4_device_status(reset=True)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("counts", [[3, 0, 20], [60, 0, 90, 7], [300, 0, 290]], ids=["32 rows", "single CTAs", "pairs"])
def test_an_early_product_waits_for_the_work_ahead_without_a_limit(early, limit, counts, gated):
    p = Grouped(counts, 608, 4096, halves=2 if gated else 1, seed=1, spread=1)
    want = [host(t.view(torch.int16)) for t in (p.swiglu() if gated else (p.gemm(),))]
    for hold in (0, HOLD):
        if gated:
            D = torch.full((p.rows, p.N // 2), 0xEE, dtype=torch.uint8, device="cuda")
            S = torch.full((mx.mxfp4_group_scale_size(p.rows, p.E, p.N),), 0xDD, dtype=torch.uint8, device="cuda")
            outs = (D, S)
        else:
            D = torch.full((p.rows, p.N), 7.0, dtype=torch.bfloat16, device="cuda")
            S, outs = None, (D,)
        torch.cuda.synchronize()
        status = early(D.data_ptr(), p.N, S.data_ptr() if gated else None, p.dA.data_ptr(), p.lda, p.dSA.data_ptr(), p.dB.data_ptr(), p.ldb,
                       (2 if gated else 1) * p.N * p.ldb, p.dSB.data_ptr(), p.dO.data_ptr(), p.E, p.rows, p.N, p.K, 0 if gated else -1,
                       hold, torch.cuda.current_stream().cuda_stream)
        assert status == 0
        torch.cuda.synchronize()
        assert mx.mxfp4_device_status() == 0, f"a wait ran out behind {hold} cycles of other work"
        for got, expect in zip(outs, want):
            np.testing.assert_array_equal(host(got.view(torch.int16)), expect)
