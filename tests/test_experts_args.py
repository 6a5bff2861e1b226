"""What the expert-layer entries accept and refuse at the ends of their ranges
(host-side checks, before any device call; no GPU)."""
import pytest

import block_scaled_mxfp4_gb300 as mx
from block_scaled_mxfp4_gb300 import build as mxbuild


@pytest.fixture(scope="module", autouse=True)
def _built():
    mxbuild.build()


P = 1 << 20                                              # a well-aligned address nothing follows


def status(call, **args):
    try:
        call(**args, stream=0)
    except mx.Mxfp4Error as e:
        return mx.STATUS_NAMES[e.status][len("MXFP4_"):]
    return "OK"


def join(**changes):
    args = dict(H=P, ldh=64, Nrm=P, ldn=64, Y=P, ldy=64, rows=20, slot_row=P, gates=P, k=2, resid=P, ldr=64, w_post=P, w_pre=P,
                res_scale=1.0, out_scale=1.0, eps=1e-6, T=10, N=64)
    return status(mx.mxfp4_moe_combine, **dict(args, **changes))


def test_a_join_without_rows_needs_no_rows():
    """Every slot is -1 then: Y is not looked at (an empty tensor's pointer is null)."""
    for changes in (dict(rows=0, Y=None), dict(rows=0, Y=None, ldy=0), dict(rows=0)):
        assert join(**changes) not in ("ERR_INVALID_ARG", "ERR_MISALIGNED")
    assert join(rows=1, Y=None) == join(rows=20, ldy=60) == "ERR_INVALID_ARG"
    assert join(rows=0, Y=None, slot_row=None, k=1) == "ERR_INVALID_ARG"      # row t of Y for every token


def test_counts_beside_the_end_of_32_bits():
    """The kernels step past the last row or token in 32 bits (a tile, or a grid of tokens): counts
    that this would carry over the end are refused."""
    last = (1 << 31) - 1
    for T in (last, last - 4864, last - 65535):
        assert join(T=T) == join(T=T, rows=T, slot_row=None, k=1) == "ERR_UNSUPPORTED_SHAPE"
    product = dict(A=P, lda=64, SA=P, B=P, ldb=64, SB=P, offsets=P, groups=4, K=64, alpha=1.0, workspace=None, workspace_bytes=0)
    for rows in (last, last - 255, last - 65535):
        assert status(mx.mxfp4_grouped_gemm, D=P, ldd=64, N=64, stride_b=4096, rows=rows, **product) == "ERR_UNSUPPORTED_SHAPE"
        assert status(mx.mxfp4_grouped_swiglu, H=P, ldh=64, SH=P, F=64, stride_b=8192, rows=rows, **product) == "ERR_UNSUPPORTED_SHAPE"
    assert join(T=last - 65536) not in ("ERR_UNSUPPORTED_SHAPE", "ERR_INVALID_ARG")
    block = dict(H=P, ldh=64, Nrm=P, ldn=64, X=P, ldx=64, ids=P, gates=P, offsets=P, slot_row=P, E=4, k=2, K=64, F=96, B1=P, ldb1=64, SB1=P,
                 B2=P, ldb2=96, SB2=P, resid=P, ldr=64, w_post=None, w_pre=None, res_scale=1.0, out_scale=1.0, eps=1e-6,
                 workspace=P, workspace_bytes=1 << 62)
    assert status(mx.mxfp4_moe_ffn, T=last // 2, **block) == "ERR_UNSUPPORTED_SHAPE"
    # The longest row of a join.
    wide = {name: 32800 for name in ("ldh", "ldn", "ldx", "ldr", "K", "ldb1")}
    assert status(mx.mxfp4_moe_ffn, T=10, **dict(block, **wide)) == "ERR_UNSUPPORTED_SHAPE"
