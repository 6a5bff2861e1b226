"""What dense_block, dense_block_backward and mxfp8_forms refuse.  No GPU: tensors on
the CPU, whose place is looked at last."""
import pytest

import block_scaled_mxfp4_gb300 as mx
from block_scaled_mxfp4_gb300 import build as mxbuild

torch = pytest.importorskip("torch")

T, K, F = 10, 64, 96


@pytest.fixture(scope="module", autouse=True)
def _built():
    mxbuild.build()


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def forward_args(packed=False):
    per = 2 if packed else 1
    return dict(x=bf16(T, K), w1=u8(F, K // per), s1=u8(F, K // 32), w2=u8(K, F // per), s2=u8(K, F // 32), b1=bf16(F), b2=bf16(K),
                norm_w=torch.zeros(K), norm_b=torch.zeros(K))


def backward_args():
    kept = mx.DenseKept(bf16(T, K), torch.zeros(K), torch.zeros(T), torch.zeros(T), u8(K, 32), u8(K, 1), u8(T, F), u8(T, F // 32),
                        mx.MXFP4_ACT_SILU, mx.MXFP8_E4M3)
    return dict(dout=bf16(T, K), kept=kept, w1t=u8(K, F), s1t=u8(K, F // 32), w2t=u8(F, K), s2t=u8(F, K // 32))


def refusal(call, args, **changes):
    for name, change in changes.items():
        args[name] = change(args[name]) if callable(change) else change
    with pytest.raises((TypeError, ValueError)) as e:
        call(**args)
    return e.type, str(e.value)


def apart(t):
    wide = torch.zeros((*t.shape, 2), dtype=t.dtype)
    wide[..., 0] = t
    return wide[..., 0]


HERE = "everything on one GPU expected"


def test_right_arguments_are_refused_for_their_place_alone():
    for packed in (False, True):
        good = lambda **c: refusal(mx.dense_block, forward_args(packed), **c)
        assert good() == (ValueError, "dense_block: " + HERE)
        assert good(b1=None, b2=None, norm_w=None, norm_b=None) == (ValueError, "dense_block: " + HERE)
        assert good(b1=lambda t: t.float(), norm_w=lambda t: t.bfloat16(), norm_b=lambda t: t.bfloat16()) == (ValueError, "dense_block: " + HERE)
        assert good(x=bf16(T, K + 5)[:, :K]) == (ValueError, "dense_block: " + HERE)      # rows may be apart
        assert good(x=bf16(0, K)) == (ValueError, "dense_block: " + HERE)
        assert good(x=torch.empty_strided((1, K), (1, 1), dtype=torch.bfloat16)) == (ValueError, "dense_block: " + HERE)
    assert refusal(mx.dense_block_backward, backward_args()) == (ValueError, "dense_block_backward: " + HERE)
    assert refusal(mx.mxfp8_forms, dict(x=bf16(3, 8))) == (ValueError, "mxfp8_forms: " + HERE)


@pytest.mark.parametrize("name,bad", [("x", torch.float16), ("x", torch.float32), ("w1", torch.bfloat16), ("s1", torch.int32),
                                      ("w2", torch.float32), ("s2", torch.int16), ("b1", torch.float16), ("b2", torch.float64),
                                      ("norm_w", torch.float64), ("norm_b", torch.bfloat16), ("norm_b", torch.int32)])
def test_types(name, bad):
    kind, text = refusal(mx.dense_block, forward_args(), **{name: lambda t: t.to(bad)})
    assert kind is TypeError and name in text


@pytest.mark.parametrize("name", ["x", "w1", "s1", "w2", "s2", "b1", "b2", "norm_w", "norm_b"])
def test_layouts(name):
    kind, text = refusal(mx.dense_block, forward_args(), **{name: apart})
    assert kind is ValueError and name in text


@pytest.mark.parametrize("name,cut", [("x", lambda t: t[:, :32]), ("x", lambda t: t[0]), ("x", lambda t: t[:1].expand(T, K)),
                                      ("w1", lambda t: t[:, :48]), ("w1", lambda t: t.t()), ("w2", lambda t: t[:, :64]),
                                      ("w2", lambda t: t[:48]), ("s1", lambda t: t[:, :1]), ("s2", lambda t: t[:, :2]),
                                      ("b1", lambda t: t[:95]), ("b2", lambda t: t[:, None]), ("norm_w", lambda t: t[:63]),
                                      ("norm_b", lambda t: t[None])])
def test_shapes(name, cut):
    kind, text = refusal(mx.dense_block, forward_args(), **{name: cut})
    assert kind is ValueError and (name in text or "w1" in text)


def test_sizes_and_codes():
    for K_, F_ in ((48, 96), (64, 80)):
        args = dict(forward_args(), x=bf16(T, K_), w1=u8(F_, K_), s1=u8(F_, K_ // 32), w2=u8(K_, F_), s2=u8(K_, F_ // 32), b1=None, b2=None,
                    norm_w=None, norm_b=None)
        assert refusal(mx.dense_block, args) == (ValueError, "dense_block: K and F multiples of 32 expected")
    for bad in (-1, 5, 99):
        assert "act" in refusal(mx.dense_block, forward_args(), act=bad)[1]
    for bad in (-1, 2, mx.MXFP6_E2M3, mx.MXFP4_E2M1_PADDED):
        assert "formats" in refusal(mx.dense_block, forward_args(), fmt=bad)[1]
        assert "formats" in refusal(mx.dense_block_backward, backward_args(), fmt_grad=bad)[1]
        assert "formats" in refusal(mx.mxfp8_forms, dict(x=bf16(3, 8)), fmt=bad)[1]
    assert "keep" in refusal(mx.dense_block, forward_args(packed=True), keep=True)[1]


@pytest.mark.parametrize("name,bad,kind", [("dout", lambda t: t.float(), TypeError), ("dout", lambda t: t[:9], ValueError),
                                           ("dout", apart, ValueError), ("dout", bf16(T, K + 4)[:, :K], ValueError),
                                           ("dout", bf16(T, K + 8)[:, 4:K + 4], ValueError),
                                           ("w1t", lambda t: t.t(), ValueError), ("w2t", lambda t: t.bfloat16(), TypeError),
                                           ("s1t", lambda t: t[:, :1], ValueError), ("s2t", lambda t: t[:90], ValueError)])
def test_gradients_arguments(name, bad, kind):
    got, text = refusal(mx.dense_block_backward, backward_args(), **{name: bad})
    assert got is kind and name in text


def test_forms_arguments():
    for bad, kind in ((bf16(3, 8).float(), TypeError), (bf16(8), ValueError), (bf16(3, 12)[:, :8], ValueError), (bf16(0, 8), ValueError),
                      (bf16(8, 8).t(), ValueError), (bf16(3, 20)[:, 4:12], ValueError)):
        with pytest.raises(kind) as e:
            mx.mxfp8_forms(bad)
        assert "GPU" not in str(e.value)
    with pytest.raises(ValueError, match="at least one form"):
        mx.mxfp8_forms(bf16(3, 8), rows=False, columns=False)


KEPT = [("x", lambda t: t.float(), TypeError), ("x", lambda t: t[0], ValueError), ("x", apart, ValueError), ("x", lambda t: t[:9], ValueError),
        ("x", lambda t: bf16(T, K + 32), ValueError), ("x", lambda t: bf16(T, 48), ValueError), ("x", lambda t: bf16(T, 0), ValueError),
        ("norm_w", lambda t: t[:63], ValueError), ("norm_w", lambda t: t.double(), TypeError),
        ("mean", lambda t: t[:9], ValueError), ("mean", lambda t: t.bfloat16(), TypeError), ("mean", apart, ValueError),
        ("rstd", lambda t: t[:, None], ValueError), ("rstd", lambda t: t.double(), TypeError), ("rstd", lambda t: t[:0], ValueError),
        ("yt", lambda t: t[:, :16], ValueError), ("yt", lambda t: t[:63], ValueError), ("yt", lambda t: t.to(torch.int16), TypeError),
        ("yt", lambda t: t.t(), ValueError), ("syt", lambda t: t[:1], ValueError), ("syt", apart, ValueError),
        ("z", lambda t: t[:9], ValueError), ("z", lambda t: t[0], ValueError), ("z", lambda t: t[:, :64], ValueError),
        ("z", lambda t: t[:, :95], ValueError), ("z", lambda t: t.float(), TypeError), ("z", lambda t: t[:, :0], ValueError),
        ("sz", lambda t: t[:, :2], ValueError), ("sz", lambda t: t[:9], ValueError), ("sz", lambda t: t.int(), TypeError)]


@pytest.mark.parametrize("name,change,kind", KEPT)
def test_what_the_forward_pass_kept(name, change, kind):
    """The kernels take each array's size from the others': one that is too short would be read past its end."""
    args = backward_args()
    args["kept"] = args["kept"]._replace(**{name: change(getattr(args["kept"], name))})
    got, text = refusal(mx.dense_block_backward, args)
    assert got is kind and HERE not in text and text.startswith("dense_block_backward: ")


def test_what_the_forward_pass_kept_with_other_codes():
    for field, bad in (("act", -1), ("act", 5), ("fmt", 2), ("fmt", mx.MXFP4_E2M1_PADDED)):
        args = backward_args()
        args["kept"] = args["kept"]._replace(**{field: bad})
        assert HERE not in refusal(mx.dense_block_backward, args)[1]


E4M3, E5M2, E8M0 = torch.float8_e4m3fn, torch.float8_e5m2, torch.float8_e8m0fnu


@pytest.mark.parametrize("fmt,right,wrong", [(mx.MXFP8_E4M3, E4M3, E5M2), (mx.MXFP8_E5M2, E5M2, E4M3)])
def test_codes_of_a_type_are_those_of_the_format(fmt, right, wrong):
    """Weights that say what their codes are: read as the other format's they would give other numbers."""
    args = dict(forward_args(), fmt=fmt)
    for name in ("w1", "w2"):
        assert refusal(mx.dense_block, dict(args), **{name: lambda t: t.view(right)})[1] == "dense_block: " + HERE
        for bad in (wrong, E8M0, torch.float8_e4m3fnuz):
            kind, text = refusal(mx.dense_block, dict(args), **{name: lambda t: t.view(bad)})
            assert kind is TypeError and name in text
    for name in ("s1", "s2"):
        assert refusal(mx.dense_block, dict(args), **{name: lambda t: t.view(E8M0)})[1] == "dense_block: " + HERE
        for bad in (E4M3, E5M2):
            kind, text = refusal(mx.dense_block, dict(args), **{name: lambda t: t.view(bad)})
            assert kind is TypeError and name in text
    args = dict(backward_args())
    args["kept"] = args["kept"]._replace(fmt=fmt)
    for name in ("w1t", "w2t"):
        assert refusal(mx.dense_block_backward, dict(args), **{name: lambda t: t.view(right)})[1] == "dense_block_backward: " + HERE
        kind, text = refusal(mx.dense_block_backward, dict(args), **{name: lambda t: t.view(wrong)})
        assert kind is TypeError and name in text
    for name, good, bad in (("yt", right, wrong), ("z", right, wrong), ("syt", E8M0, right), ("sz", E8M0, right)):
        put = lambda to: dict(args, kept=args["kept"]._replace(**{name: getattr(args["kept"], name).view(to)}))
        assert refusal(mx.dense_block_backward, put(good))[1] == "dense_block_backward: " + HERE
        kind, text = refusal(mx.dense_block_backward, put(bad))
        assert kind is TypeError and "kept." + name in text


def test_packed_codes_of_a_type():
    for name in ("w1", "w2"):
        assert refusal(mx.dense_block, forward_args(packed=True), **{name: lambda t: t.view(torch.float4_e2m1fn_x2)})[1] == "dense_block: " + HERE
        for bad in (E4M3, E5M2, E8M0):
            kind, text = refusal(mx.dense_block, forward_args(packed=True), **{name: lambda t: t.view(bad)})
            assert kind is TypeError and name in text


def test_rows_longer_than_the_norms():
    for K_, text in ((32768, HERE), (32800, "K of at most 32768 expected")):
        args = dict(forward_args(), x=bf16(2, K_), w1=u8(32, K_), s1=u8(32, K_ // 32), w2=u8(K_, 32), s2=u8(K_, 1), b1=None, b2=None,
                    norm_w=None, norm_b=None)
        assert refusal(mx.dense_block, args) == (ValueError, "dense_block: " + text)
        kept = mx.DenseKept(bf16(2, K_), None, torch.zeros(2), torch.zeros(2), u8(K_, 32), u8(K_, 1), u8(2, 32), u8(2, 1), 0, 0)
        args = dict(dout=bf16(2, K_), kept=kept, w1t=u8(K_, 32), s1t=u8(K_, 1), w2t=u8(32, K_), s2t=u8(32, K_ // 32))
        assert refusal(mx.dense_block_backward, args) == (ValueError, "dense_block_backward: " + text)


def test_eps():
    assert refusal(mx.dense_block, forward_args(), eps=0)[1] == "dense_block: " + HERE
    for bad in (-1e-9, float("nan")):
        assert refusal(mx.dense_block, forward_args(), eps=bad) == (ValueError, "dense_block: eps of at least 0 expected")


def test_another_device_than_the_launches(monkeypatch):
    """Pointers to one GPU's memory are no other's to read.  No GPU: devices by name."""
    from types import SimpleNamespace

    from block_scaled_mxfp4_gb300 import dense

    class Stream:
        def __init__(self, index, handle):
            self.device, self.cuda_stream = torch.device("cuda", index), handle

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Stream(0, 0))
    on = [SimpleNamespace(is_cuda=True, device=torch.device("cuda", i)) for i in (0, 1)]

    def refused(stream, *tensors):
        try:
            dense._check_place("here", stream, *tensors)
        except ValueError as e:
            return str(e)

    assert refused(None, on[0], on[0], None) is None and refused(77, on[0]) is None
    assert refused(Stream(0, 5), on[0]) is None and refused(Stream(1, 5), on[1], on[1]) is None
    assert refused(None, on[0], on[1]) == "here: " + HERE
    # (a default stream's handle is the same on every device: nothing switches to its device)
    for stream, tensor in ((None, 1), (77, 1), (Stream(0, 5), 1), (Stream(1, 5), 0), (Stream(1, 0), 1)):
        assert "device of the current stream" in refused(stream, on[tensor])
