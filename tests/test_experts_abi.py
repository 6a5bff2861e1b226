"""Host-side checks of the expert-layer entry points that need no GPU: sizes,
refusals (before any device call) and the plain forms the GPU tests use."""
import numpy as np
import pytest

import block_scaled_mxfp4_gb300 as mx
import expert_ref as ref
from block_scaled_mxfp4_gb300 import build as mxbuild


@pytest.fixture(scope="module", autouse=True)
def _built():
    mxbuild.build()


P = 1 << 20                                              # a well-aligned address nothing follows


def status(call, *args):
    try:
        call(*args, stream=0)
    except mx.Mxfp4Error as e:
        return mx.STATUS_NAMES[e.status][len("MXFP4_"):]
    return "OK"


def change(args, **by_index):
    out = list(args)
    for k, v in by_index.items():
        out[int(k[1:])] = v
    return out


ROUTE = [P, P, P, P, P, P, 64, 0, None, 100, 64, 4, 0, 1.0, P, 1 << 20]
QUANT = [P, 64, P, P, 64, 10, 64, P, P, 2, P, 4, 20]
GEMM = [P, 64, P, 64, P, P, 64, 64 * 64, P, P, 4, 10, 64, 64, 1.0, P, 1 << 28]
GATED = [P, 64, P, P, 64, P, P, 64, 2 * 64 * 64, P, P, 4, 10, 64, 64, 1.0, P, 1 << 28]
JOIN = [P, 64, P, 64, P, 64, 20, P, P, 2, P, 64, P, P, 1.0, 1.0, 1e-6, 10, 64]
FFN = [P, 64, P, 64, P, 64, P, P, P, P, 10, 4, 2, 64, 96, P, 64, P, P, 96, P, P, 64, None, None, 1.0, 1.0, 1e-6, P, 1 << 30]

REFUSALS = [
    (mx.mxfp4_moe_route, ROUTE, [(dict(_0=None), "ERR_INVALID_ARG"), (dict(_2=None), "ERR_INVALID_ARG"),
                                 (dict(_6=63), "ERR_INVALID_ARG"), (dict(_7=2), "ERR_INVALID_ARG"),
                                 (dict(_9=-1), "ERR_INVALID_ARG"), (dict(_10=0), "ERR_INVALID_ARG"),
                                 (dict(_10=1025, _6=2000), "ERR_INVALID_ARG"), (dict(_11=0), "ERR_INVALID_ARG"),
                                 (dict(_11=17), "ERR_INVALID_ARG"), (dict(_10=3), "ERR_INVALID_ARG"),
                                 (dict(_12=3), "ERR_INVALID_ARG"), (dict(_5=P + 1), "ERR_MISALIGNED"),
                                 (dict(_5=P + 2, _7=1), "ERR_MISALIGNED"), (dict(_14=None), "ERR_WORKSPACE"),
                                 (dict(_15=16), "ERR_WORKSPACE"), (dict(_14=P + 16), "ERR_MISALIGNED"),
                                 (dict(_9=1 << 30), "ERR_UNSUPPORTED_SHAPE")]
     + [({f"_{i}": P + 2}, "ERR_MISALIGNED") for i in range(5)]),
    (mx.mxfp4_group_quantize, QUANT, [(dict(_0=None), "ERR_INVALID_ARG"), (dict(_10=None), "ERR_INVALID_ARG"),
                                      (dict(_6=48), "ERR_INVALID_ARG"), (dict(_4=32), "ERR_INVALID_ARG"),
                                      (dict(_8=None), "ERR_INVALID_ARG"), (dict(_9=0), "ERR_INVALID_ARG"),
                                      (dict(_9=17), "ERR_INVALID_ARG"), (dict(_7=None, _8=None), "ERR_INVALID_ARG"),
                                      (dict(_7=None, _8=None, _9=1), "ERR_INVALID_ARG"),
                                      (dict(_11=0), "ERR_INVALID_ARG"), (dict(_1=80), "ERR_MISALIGNED"),
                                      (dict(_3=P + 2), "ERR_MISALIGNED"), (dict(_2=P + 4), "ERR_MISALIGNED")]
     + [({f"_{i}": P + 2}, "ERR_MISALIGNED") for i in (7, 8, 10)]),
    (mx.mxfp8_group_quantize, QUANT + [mx.MXFP8_E4M3], [(dict(_13=mx.MXFP6_E2M3), "ERR_INVALID_ARG"),
                                                        (dict(_1=72), "ERR_MISALIGNED")]),
    (mx.mxfp4_grouped_gemm, GEMM, [(dict(_0=None), "ERR_INVALID_ARG"), (dict(_9=None), "ERR_INVALID_ARG"),
                                   (dict(_1=63), "ERR_INVALID_ARG"), (dict(_3=32), "ERR_INVALID_ARG"),
                                   (dict(_7=64 * 63), "ERR_INVALID_ARG"), (dict(_10=1025), "ERR_INVALID_ARG"),
                                   (dict(_11=-1), "ERR_INVALID_ARG"), (dict(_12=0), "ERR_INVALID_ARG"),
                                   (dict(_13=40), "ERR_INVALID_ARG"), (dict(_3=80), "ERR_MISALIGNED"),
                                   (dict(_2=P + 8), "ERR_MISALIGNED"), (dict(_7=64 * 64 + 16), "ERR_MISALIGNED"),
                                   (dict(_8=P + 8), "ERR_MISALIGNED"), (dict(_0=P + 1), "ERR_MISALIGNED"),
                                   (dict(_9=P + 2), "ERR_MISALIGNED"),
                                   (dict(_11=(1 << 31) - 1, _12=1 << 30, _1=1 << 30, _7=1 << 40),
                                    "ERR_UNSUPPORTED_SHAPE")]),
    (mx.mxfp8_grouped_gemm, GEMM[:14] + [0, 1] + GEMM[14:], [(dict(_14=2), "ERR_INVALID_ARG"),
                                                             (dict(_15=6), "ERR_INVALID_ARG")]),
    (mx.mxfp4_grouped_swiglu, GATED, [(dict(_2=None), "ERR_INVALID_ARG"), (dict(_13=48), "ERR_INVALID_ARG"),
                                      (dict(_8=64 * 64), "ERR_INVALID_ARG"), (dict(_1=80), "ERR_MISALIGNED"),
                                      (dict(_0=P + 8), "ERR_MISALIGNED"), (dict(_2=P + 8), "ERR_MISALIGNED")]),
    (mx.mxfp8_grouped_swiglu, GATED[:15] + [0, 0, 0] + GATED[15:], [(dict(_17=3), "ERR_INVALID_ARG"),
                                                                    (dict(_15=2), "ERR_INVALID_ARG")]),
    (mx.mxfp4_moe_combine, JOIN, [(dict(_0=None, _2=None), "ERR_INVALID_ARG"), (dict(_4=None), "ERR_INVALID_ARG"),
                                  (dict(_1=60), "ERR_INVALID_ARG"), (dict(_11=60), "ERR_INVALID_ARG"),
                                  (dict(_7=None), "ERR_INVALID_ARG"), (dict(_7=None, _9=1, _6=9), "ERR_INVALID_ARG"),
                                  (dict(_9=17), "ERR_INVALID_ARG"), (dict(_16=-1.0), "ERR_INVALID_ARG"),
                                  (dict(_16=float("nan")), "ERR_INVALID_ARG"), (dict(_4=P + 1), "ERR_MISALIGNED"),
                                  (dict(_7=P + 2), "ERR_MISALIGNED"), (dict(_8=P + 2), "ERR_MISALIGNED"),
                                  (dict(_18=40000, _1=40000, _3=40000, _5=40000, _11=40000),
                                   "ERR_UNSUPPORTED_SHAPE")]),
    (mx.mxfp4_moe_ffn, FFN, [(dict(_6=None), "ERR_INVALID_ARG"), (dict(_8=None), "ERR_INVALID_ARG"),
                             (dict(_0=None, _2=None), "ERR_INVALID_ARG"), (dict(_12=5), "ERR_INVALID_ARG"),
                             (dict(_14=48), "ERR_INVALID_ARG"), (dict(_16=32), "ERR_INVALID_ARG"),
                             (dict(_18=None), "ERR_INVALID_ARG"), (dict(_29=1000), "ERR_WORKSPACE"),
                             (dict(_28=None), "ERR_WORKSPACE"), (dict(_28=P + 8), "ERR_MISALIGNED"),
                             (dict(_4=P + 2), "ERR_MISALIGNED"),
                             *[({f"_{i}": P + 2}, "ERR_MISALIGNED") for i in (6, 7, 8, 9)], (dict(_13=32800, _5=32800), "ERR_INVALID_ARG")]),
]


@pytest.mark.parametrize("call,args,changes", REFUSALS, ids=lambda v: getattr(v, "__name__", ""))
def test_refusals(call, args, changes):
    for by, want in changes:
        assert status(call, *change(args, **by)) == want, (call.__name__, by)


def test_sizes():
    assert mx.mxfp4_group_scale_size(0, 3, 32) == 3 * 1024
    assert mx.mxfp4_group_scale_size(256, 8, 512) == 10 * 4 * 512
    assert mx.mxfp4_group_scale_size(10, 0, 32) == mx.mxfp4_group_scale_size(10, 1, 31) == 0
    assert mx.mxfp4_moe_route_workspace_size(64, 128) == 0
    assert mx.mxfp4_moe_route_workspace_size(10 ** 6, 128) <= 152 * 128 * 2
    assert mx.mxfp4_moe_route_workspace_size(-1, 128) == 0
    whole = mx.mxfp4_moe_ffn_workspace_size(100, 8, 2, 512, 256)
    parts = 200 * (256 + 128 + 1024) + mx.mxfp4_group_scale_size(200, 8, 512) + mx.mxfp4_group_scale_size(200, 8, 256)
    assert whole >= parts
    assert mx.mxfp4_moe_ffn_workspace_size(100, 8, 9, 512, 256) == 0


def test_the_grouped_scale_layout_never_overlaps():
    """Blocks of the layout: every group's start after its predecessor's end, inside the size."""
    rng = np.random.default_rng(0)
    for _ in range(200):
        counts = rng.integers(0, 400, size=rng.integers(1, 30)) * (rng.uniform(size=1) < 0.8)
        counts = np.where(rng.uniform(size=counts.size) < 0.3, 0, counts)
        offsets = np.concatenate([[0], np.cumsum(counts)])
        at = ref.scale_places(offsets, 64)
        assert len(np.unique(at)) == at.size
        if at.size:
            assert at.max() < mx.mxfp4_group_scale_size(int(offsets[-1]), len(counts), 64)


def test_plain_quantiser_agrees_with_the_oracle(oracle_mod):
    """The plain form's rounding is the oracle quantisers' (which the dense quantisers are held to)."""
    rng = np.random.default_rng(1)
    x = (rng.normal(size=(40, 256)) * np.exp(3 * rng.normal(size=(40, 256)))).astype(np.float32)
    bits = (x.view(np.uint32) >> 16).astype(np.uint16)     # truncated: any bf16 will do
    v = (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    for fmt, call in (("e2m1", lambda: oracle_mod.quantize(bits, 40, 256)), ("e4m3", lambda: oracle_mod.quantize8(bits, 40, 256, oracle_mod.E4M3)),
                      ("e5m2", lambda: oracle_mod.quantize8(bits, 40, 256, oracle_mod.E5M2))):
        codes, scales = ref.quantise(v, fmt)
        q, s = call()[:2]
        np.testing.assert_array_equal(codes, q.reshape(codes.shape))
        np.testing.assert_array_equal(scales, s.reshape(scales.shape))


@pytest.mark.parametrize("call,args,changes", REFUSALS, ids=lambda v: getattr(v, "__name__", ""))
def test_refusals_through_the_bound_entries(call, args, changes):
    """Loading the library puts the extension module's functions in place of
    the Python ones: the same refusals, stream by place or by name."""
    mx.lib()
    bound = getattr(mx, call.__name__)
    assert bound is not call and type(bound).__name__ == "builtin_function_or_method"
    for by, want in changes:
        assert status(bound, *change(args, **by)) == want, (call.__name__, by)
        with pytest.raises(mx.Mxfp4Error) as e:
            bound(*change(args, **by), 0)
        assert want in str(e.value) and call.__name__ in str(e.value)


def test_the_bound_entries_check_their_arguments():
    mx.lib()
    good = change(JOIN, _18=0)                            # refused by the library, once converted
    with pytest.raises(TypeError):
        mx.mxfp4_moe_combine(*good[:-1], stream=0)
    with pytest.raises(TypeError):
        mx.mxfp4_moe_combine(*good, flow=0)
    with pytest.raises(TypeError):
        mx.mxfp4_moe_combine(*change(good, _4="Y"), stream=0)
    with pytest.raises(TypeError):
        mx.mxfp4_moe_combine(*change(good, _14="1.0"), stream=0)
    with pytest.raises(OverflowError):
        mx.mxfp4_moe_combine(*change(good, _17=1 << 40), stream=0)
    with pytest.raises(OverflowError):
        mx.mxfp4_moe_route(*change(ROUTE, _15=-1), stream=0)

    class Stream:
        cuda_stream = 0

    class Pointer:
        def data_ptr(self):
            return P

    with pytest.raises(mx.Mxfp4Error):
        mx.mxfp4_moe_combine(*change(good, _4=Pointer(), _0=np.zeros(8)), Stream())
