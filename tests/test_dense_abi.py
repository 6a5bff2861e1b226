"""Host-side checks of the dense layer's entry points that need no GPU: the
lists of their arguments agree, sizes, refusals (before any device call)."""
import ctypes
import inspect
import re

import pytest

import block_scaled_mxfp4_gb300 as mx
from block_scaled_mxfp4_gb300 import build as mxbuild

ENTRIES = ["mxfp4_gemm_act", "mxfp8_gemm_act", "mxfp8_checkpoint", "mxfp8_act_backward", "mxfp4_layer_norm", "mxfp4_layer_norm_backward"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    mxbuild.build()
    mx.lib()


P = 1 << 20                                              # a well-aligned address nothing follows
LAST = (1 << 31) - 1


def status(call, **args):
    try:
        call(**args, stream=0)
    except mx.Mxfp4Error as e:
        return mx.STATUS_NAMES[e.status][len("MXFP4_"):]
    return "OK"


def passes(call, **args):
    """Nothing about the arguments is refused (without a GPU the call ends at the device's check)."""
    return status(call, **args) in ("OK", "ERR_CUDA", "ERR_ARCH")


PRODUCT = dict(D=P, ldd=64, H=P, ldh=64, SH=P, ld_sh=2, Z=P, ldz=64, SZ=P, ld_sz=2, A=P, lda=96, B=P, ldb=96, scaleA=P, ld_sa=3, scaleB=P,
               ld_sb=3, fmt_z=0, alpha=1.0, bias=P, bias_type=0, act=2, R=P, ldr=64, res_scale=1.0, M=10, N=64, K=96, split_k=0, flags=0,
               workspace=None, workspace_bytes=0)
BYTES = dict(PRODUCT, fmt_a=0, fmt_b=1, fmt_h=0)
CHECKPOINT = dict(Q=P, ldq=96, S=P, lds=3, QT=P, ldqt=64, ST=P, ldst=2, col_sums=P, X=P, ldx=80, rows=50, cols=75, fmt=0, workspace=P,
                  workspace_bytes=1 << 40)
BACKWARD = dict(dZ=P, lddz=75, Q=P, ldq=96, S=P, lds=3, QT=P, ldqt=64, ST=P, ldst=2, HT=P, ldht=64, SHT=P, ld_sht=2, dbias=P, dH=P, lddh=80,
                Z=P, ldz=96, SZ=P, ld_sz=3, fmt_z=0, act=4, rows=50, cols=75, fmt=1, fmt_h=0, workspace=P, workspace_bytes=1 << 40)
NORM = dict(Y=P, ldy=75, mean=P, rstd=P, X=P, ldx=75, w=P, b=P, param_type=0, eps=1e-5, T=50, N=75)
NORM_GRAD = dict(dX=P, lddx=75, dw=P, db=P, dY=P, lddy=75, X=P, ldx=75, mean=P, rstd=P, w=P, param_type=1, dres=P, ldr=75, T=50, N=75,
                 workspace=P, workspace_bytes=1 << 40)

INVALID, MISALIGNED, SHAPE, WORKSPACE = "ERR_INVALID_ARG", "ERR_MISALIGNED", "ERR_UNSUPPORTED_SHAPE", "ERR_WORKSPACE"
OUTPUTS = [dict(H=None), dict(SH=None), dict(ldh=32), dict(ld_sh=1), dict(Z=None), dict(SZ=None), dict(ldz=32), dict(ld_sz=1), dict(fmt_z=2),
           dict(fmt_z=3), dict(act=-1), dict(act=5), dict(bias_type=2), dict(ldr=63), dict(flags=2), dict(ldd=63), dict(A=None), dict(B=None),
           dict(scaleA=None), dict(ld_sb=2), dict(M=0), dict(N=0), dict(K=48), dict(K=0), dict(split_k=17), dict(split_k=-1),
           dict(N=63), dict(D=None, H=None, SH=None, Z=None, SZ=None)]
APART = [dict(A=P + 8), dict(lda=104), dict(Z=P + 8), dict(ldz=72), dict(H=P + 8), dict(D=P + 1), dict(R=P + 1), dict(bias=P + 1),
         dict(bias=P + 2, bias_type=1), dict(workspace=P + 16)]
REFUSALS = {
    "mxfp4_gemm_act": (PRODUCT, {INVALID: OUTPUTS, MISALIGNED: APART + [dict(ldh=80)]}),
    "mxfp8_gemm_act": (BYTES, {INVALID: OUTPUTS + [dict(fmt_a=2), dict(fmt_b=6), dict(fmt_h=2), dict(fmt_h=5)],
                               MISALIGNED: APART + [dict(ldh=72)]}),
    "mxfp8_checkpoint": (CHECKPOINT, {
        INVALID: [dict(Q=None), dict(S=None), dict(QT=None), dict(ST=None), dict(ldq=80), dict(lds=2), dict(ldqt=48), dict(ldst=1), dict(X=None),
                  dict(ldx=72), dict(rows=0), dict(cols=0), dict(rows=-1), dict(fmt=2), dict(fmt=3),
                  dict(Q=None, S=None, QT=None, ST=None, col_sums=None)],
        MISALIGNED: [dict(Q=P + 8), dict(ldq=104), dict(QT=P + 8), dict(ldqt=72), dict(X=P + 8), dict(ldx=81), dict(col_sums=P + 2)],
        SHAPE: [dict(rows=LAST, ldqt=1 << 31, ldst=1 << 26), dict(cols=LAST, ldq=1 << 31, lds=1 << 26, ldx=1 << 31)]}),
    "mxfp8_act_backward": (BACKWARD, {
        INVALID: [dict(Q=None), dict(S=None), dict(QT=None), dict(ST=None), dict(HT=None), dict(SHT=None), dict(ldq=80), dict(ldqt=48),
                  dict(ldht=48), dict(ld_sht=1), dict(lddz=74), dict(dH=None), dict(lddh=72), dict(Z=None), dict(SZ=None), dict(ldz=80),
                  dict(ld_sz=2), dict(fmt_z=3), dict(fmt=4), dict(fmt_h=5), dict(act=5), dict(act=-1), dict(rows=0), dict(cols=0),
                  dict(dZ=None, Q=None, S=None, QT=None, ST=None, HT=None, SHT=None, dbias=None)],
        MISALIGNED: [dict(Z=P + 8), dict(ldz=104), dict(dH=P + 2), dict(lddh=81), dict(HT=P + 4), dict(ldht=72), dict(dZ=P + 1), dict(dbias=P + 1)],
        SHAPE: [dict(rows=LAST, ldqt=1 << 31, ldst=1 << 26, ldht=1 << 31, ld_sht=1 << 26)]}),
    "mxfp4_layer_norm": (NORM, {
        INVALID: [dict(Y=None), dict(X=None), dict(ldy=74), dict(ldx=74), dict(param_type=2), dict(param_type=-1), dict(eps=-1e-9),
                  dict(eps=float("nan")), dict(T=-1), dict(N=0)],
        MISALIGNED: [dict(Y=P + 1), dict(X=P + 1), dict(mean=P + 2), dict(rstd=P + 2), dict(w=P + 1), dict(b=P + 2, param_type=1)],
        SHAPE: [dict(N=32769, ldx=40000, ldy=40000), dict(T=LAST)]}),
    "mxfp4_layer_norm_backward": (NORM_GRAD, {
        INVALID: [dict(dX=None), dict(dY=None), dict(X=None), dict(mean=None), dict(rstd=None), dict(lddx=74), dict(lddy=74), dict(ldx=74),
                  dict(ldr=74), dict(param_type=2), dict(T=-1), dict(N=0)],
        MISALIGNED: [dict(dX=P + 1), dict(dY=P + 1), dict(X=P + 1), dict(dres=P + 1), dict(mean=P + 2), dict(dw=P + 2), dict(db=P + 1),
                     dict(w=P + 2), dict(workspace=P + 64)],
        SHAPE: [dict(N=32769, ldx=40000, lddx=40000, lddy=40000, ldr=40000), dict(T=LAST)],
        WORKSPACE: [dict(workspace=None), dict(workspace_bytes=8)]}),
}


@pytest.mark.parametrize("name", ENTRIES)
def test_refusals(name):
    good, bad = REFUSALS[name]
    call = getattr(mx, name)
    assert passes(call, **good)
    for want, changes in bad.items():
        for change in changes:
            assert status(call, **dict(good, **change)) == want, (name, change)


def test_what_may_be_left_out():
    for name, groups in (("mxfp4_gemm_act", (("D",), ("H", "SH"), ("Z", "SZ"), ("bias",), ("R",))),
                         ("mxfp8_gemm_act", (("D",), ("H", "SH"), ("Z", "SZ"), ("bias",), ("R",))),
                         ("mxfp8_checkpoint", (("Q", "S"), ("QT", "ST"), ("col_sums",))),
                         ("mxfp8_act_backward", (("dZ",), ("Q", "S"), ("QT", "ST"), ("HT", "SHT"), ("dbias",))),
                         ("mxfp4_layer_norm", (("mean",), ("rstd",), ("w",), ("b",))),
                         ("mxfp4_layer_norm_backward", (("dw",), ("db",), ("w",), ("dres",)))):
        good = REFUSALS[name][0]
        for names in groups:
            assert passes(getattr(mx, name), **dict(good, **{n: None for n in names})), (name, names)
    # What the left-out arrays' strides say is not looked at, nor a workspace that nothing needs.
    assert passes(mx.mxfp4_gemm_act, **dict(PRODUCT, D=None, ldd=0, H=None, SH=None, ldh=0, ld_sh=0, R=None, ldr=0, N=63))
    assert passes(mx.mxfp8_checkpoint, **dict(CHECKPOINT, col_sums=None, workspace=None, workspace_bytes=0, rows=10 ** 6, ldqt=10 ** 6, ldst=31250))
    assert status(mx.mxfp8_checkpoint, **dict(CHECKPOINT, workspace=None, rows=10 ** 6, ldqt=10 ** 6, ldst=31250)) == WORKSPACE
    assert passes(mx.mxfp4_layer_norm_backward, **dict(NORM_GRAD, dw=None, db=None, workspace=None, workspace_bytes=0))
    # No rows: no array is touched.
    none = dict.fromkeys(("Y", "X", "mean", "rstd", "w", "b"))
    assert passes(mx.mxfp4_layer_norm, **dict(NORM, T=0, ldx=0, ldy=0, **none))
    none = dict.fromkeys(("dX", "dY", "X", "mean", "rstd", "w", "dres", "dw", "db", "workspace"))
    assert passes(mx.mxfp4_layer_norm_backward, **dict(NORM_GRAD, T=0, lddx=0, lddy=0, ldx=0, **none))


def test_sizes():
    for rows, cols in ((1, 1), (32, 64), (1000, 33), (10 ** 6, 4096), (16384, 8192)):
        a = mx.mxfp8_checkpoint_workspace_size(rows, cols)
        assert a % 256 == 0 and a <= 4 * cols * -(-rows // 32) + 256
        b = mx.mxfp4_layer_norm_workspace_size(rows, min(cols, 32768))
        assert b % 256 == 0 and b <= 8 * cols * min(rows, 1216) + 256
    assert mx.mxfp8_checkpoint_workspace_size(0, 5) == mx.mxfp8_checkpoint_workspace_size(5, 0) == mx.mxfp8_checkpoint_workspace_size(LAST, 5) == 0
    assert mx.mxfp4_layer_norm_workspace_size(-1, 5) == mx.mxfp4_layer_norm_workspace_size(5, 0) == 0
    assert mx.mxfp4_layer_norm_workspace_size(5, 32769) == 0 == mx.mxfp4_layer_norm_workspace_size(1, 32768)


def parameters(name):
    return list(inspect.signature(mx._python_entries[name]).parameters)


@pytest.mark.parametrize("name", ENTRIES)
def test_header_table_and_python_agree(name):
    python, extension = mx._python_entries[name], getattr(mx, name)
    assert type(extension).__name__ == "builtin_function_or_method" and inspect.isfunction(python)
    assert str(inspect.signature(python)) == str(inspect.signature(extension)) and python.__doc__ == extension.__doc__
    text = re.sub(r"/\*.*?\*/", "", open(mx.HEADER).read(), flags=re.S)
    declared = re.search(r"\bint\s+%s\s*\(([^)]*)\)" % name, text).group(1).split(",")
    names = [re.search(r"(\w+)\s*$", d).group(1) for d in declared]
    kinds = {"int64_t": ctypes.c_int64, "size_t": ctypes.c_size_t, "float": ctypes.c_float, "int": ctypes.c_int, "unsigned": ctypes.c_uint}
    types = [ctypes.c_void_p if "*" in d else kinds[d.replace("const", "").split()[0]] for d in declared]
    assert names == parameters(name) and types == list(getattr(mx.lib(), name).argtypes)


@pytest.mark.parametrize("form", ["python", "extension"])
@pytest.mark.parametrize("name", ENTRIES)
def test_arguments_by_place_and_name(name, form):
    call, names = (mx._python_entries[name] if form == "python" else getattr(mx, name)), parameters(name)
    values = {n: 0 for n in names}
    n = len(names)
    for by_place in (0, 1, n // 2, n - 1, n):
        with pytest.raises(mx.Mxfp4Error) as e:
            call(*list(values.values())[:by_place], **{k: values[k] for k in reversed(names[by_place:])})
        assert name in str(e.value) and e.value.status == -1
    with pytest.raises(TypeError):
        call(*[0] * (n + 1))
    if form == "extension" and "flags" in names:
        for bad in (-1, 1 << 32):
            with pytest.raises(OverflowError):
                call(**dict(values, flags=bad))
