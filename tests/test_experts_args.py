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
