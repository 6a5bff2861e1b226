"""What the header says of the dense layer's operators at the far ends of their arguments."""
import numpy as np
import pytest

import block_scaled_mxfp4_gb300 as mx
import dense_ref as dr
import expert_ref as ref
from test_gpu_dense import KIND, Product, bf16, dev, host, run_backward, workspace

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


@pytest.mark.parametrize("act", dr.ACTS)
@pytest.mark.parametrize("fmt_z", ["e4m3", "e5m2"])
def test_slopes_of_large_z(fmt_z, act):
    """z from 2^13 up to the largest fp32 numbers, which 8 bits with a scale hold: there every slope is 1 above
    zero, and 0 below (1 with no activation), to far more digits than fp32 has, and so dz is dh or 0."""
    emax, mantissas = {"e4m3": (8, 7), "e5m2": (15, 4)}[fmt_z]
    scales = np.arange(127 + 13 - emax, 255 - emax)          # of z from 2^13 to under 2^128
    rows, cols = len(scales), 96
    rng = np.random.default_rng(8)
    codes = 0x78 + rng.integers(0, mantissas, size=(rows, cols)) + 0x80 * rng.integers(0, 2, size=(rows, cols))
    codes[:, 5:9] = 0                                        # and zeros among them
    codes, s = codes.astype(np.uint8), np.repeat(scales[:, None], 3, axis=1).astype(np.uint8)
    z = ref.values(codes, s, fmt_z)
    assert np.abs(z).max() < 2.0 ** 128 and (np.abs(z[z != 0]) >= 2.0 ** 13).all()
    dh, g = bf16(rng.normal(size=(rows, cols)))
    dZ, Q, S, QT, ST, HT, SHT, db = map(host, run_backward(dh, dev(codes), dev(s), fmt_z, act, cols))
    one, zero = 1.0, (1.0 if act == "none" else 0.0)
    slope = np.where(z == 0, {"none": 1.0, "relu": 0.0}.get(act, 0.5), np.where(z > 0, one, zero))
    h, v = z if act == "none" else np.maximum(z, 0), g * slope
    e = np.where(z == 0, 2.0 ** -19 * np.abs(g), 0.0)        # exp, 1 / x and the polynomial, at 0
    dr.check_bf16(dZ, v, e, "dZ")
    dr.check_codes(Q, S, v, e, "e4m3", "rows")
    dr.check_codes(QT, ST, v.T.copy(), e.T.copy(), "e4m3", "columns")
    dr.check_codes(HT, SHT, h.T.copy(), 0, "e4m3", "h")
    # (chains of fp32 additions: a lane's rows, then lanes, warps and strips)
    assert (np.abs(db - v.sum(0)) <= (rows / 32 + 64) * dr.EPS24 * np.abs(v).sum(0) + e.sum(0)).all()


@pytest.mark.parametrize("act,lo,hi", [("silu", -130.0, 20.0), ("gelu_tanh", -14.0, 6.0), ("gelu", -15.0, 6.0), ("relu", -3.0, 3.0)])
def test_activations_down_to_the_smallest_numbers(act, lo, hi):
    """Every activation within the header's bound of its value, with nothing but what the header allows
    for small ones: 0 under the smallest normal number, or for SiLU and GELU's tanh form where the
    sigmoid is under 2^-125.  z is the bias: the product's sums are 0."""
    N = 1 << 15
    p = Product("mxfp8", 2, N, 32, 12)
    p.dA.zero_()
    z = np.linspace(lo, hi, N).astype(np.float32)
    D = host(p.run(act, dev(z), "fp32")[0])
    z = z.astype(np.float64)
    if act == "silu":
        u = z
    elif act == "gelu_tanh":
        u = np.sqrt(8 / np.pi) * (z + 0.044715 * z ** 3)
    else:
        u = z * z / 2 if act == "gelu" else 0.0 * z
    if act in ("silu", "gelu_tanh"):
        g = np.exp(u - np.logaddexp(0, u))
        h, zero = z * g, np.where(g < 2.0 ** -125, np.abs(z) * g, 0.0)
    else:
        h = dr.act(z, act)[0]
        zero = np.where(np.abs(h) < 2.0 ** -126, np.abs(h), 0.0)
    e = np.abs(h) * (2.0 ** -19 + np.abs(u) * 2.0 ** -21) if act != "relu" else 0.0
    for row in D:
        dr.check_bf16(row, h, np.maximum(e, zero), act)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("T,N", [(5, 200), (300, 200), (20, 512), (76, 1024), (77, 1024), (300, 1024), (1300, 1024), (20, 2048), (300, 2048), (3000, 1024),
                                 (40, 4096), (100, 4104), (700, 9000), (400, 17000), (33, 1022), (33, 1001)])
def test_order_of_a_norm_gradients_sums(T, N, kind):
    """Sizes and the rows' alignment decide it, not the weight's."""
    x, dy = (torch.randn((T, N), device="cuda").bfloat16() for _ in range(2))
    m, r = x.float().mean(1), 1 + torch.rand(T, device="cuda")
    base = torch.randn(N, device="cuda").to(torch.bfloat16 if kind == "bf16" else torch.float32)
    ws = workspace(mx.mxfp4_layer_norm_workspace_size(T, N))
    outs = []
    for off in (0, 1, 2, 4):
        w = torch.zeros(N + 8, dtype=base.dtype, device="cuda")
        w[off:off + N] = base
        dx, dw, db = torch.empty_like(x), torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
        mx.mxfp4_layer_norm_backward(dx, N, dw, db, dy, N, x, N, m, r, w[off:off + N], KIND[kind], None, 0, T, N, ws, ws.numel())
        outs.append((dx, dw, db))
    torch.cuda.synchronize()
    for one in outs[1:]:
        for a, b in zip(outs[0], one):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("act", dr.ACTS)
def test_columns_behind_a_block_that_is_not_finite(act):
    """The last block's columns past the last one are zeros in the forms along the rows, whatever its z."""
    rows, cols = 70, 75
    rng = np.random.default_rng(9)
    codes, s = (rng.integers(0, 0x78, size=(rows, 96)).astype(np.uint8), np.full((rows, 3), 122, np.uint8))
    s[3, 2] = s[69, 2] = 255
    s[40, 1] = 255
    dh, _ = bf16(rng.normal(size=(rows, cols)), ld=80)
    Q, S = map(host, run_backward(dh, dev(codes), dev(s), "e4m3", act, cols)[1:3])
    assert (Q[:, cols:96] == 0).all()
    if act not in ("none", "relu"):
        assert ((S[:, :3] == 255) == (s == 255)).all()


@pytest.mark.parametrize("act", dr.ACTS)
def test_slopes_of_infinite_z(act):
    rows, cols = 32, 64
    codes, s = np.full((rows, cols), 0x3C, np.uint8), np.full((rows, 2), 127, np.uint8)      # ones
    codes[3, 5], codes[7, 40] = 0x7C, 0xFC
    codes[9, 32:] = 0x7B                                     # 57344 2^127
    s[9, 1] = 254
    dh, g = bf16(np.random.default_rng(10).normal(size=(rows, cols)))
    dZ = host(run_backward(dh, dev(codes), dev(s), "e5m2", act, cols)[0])
    odd = np.zeros((rows, cols), bool)
    odd[3, 5] = odd[7, 40] = odd[9, 32:] = True
    if act in ("none", "relu"):
        want = g.copy()
        want[7, 40] *= act == "none"
        assert (dZ == want).all()
    else:
        assert (np.isnan(dZ) == odd).all()
