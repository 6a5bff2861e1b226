"""moe_block and relaid_expert_scales take tensors where the entries under them
take pointers, so they are the ones to refuse a wrong type or layout.  No GPU:
tensors on the CPU, whose place is looked at last."""
import pytest

import block_scaled_mxfp4_gb300 as mx
from block_scaled_mxfp4_gb300 import build as mxbuild

torch = pytest.importorskip("torch")

T, E, K, F = 10, 4, 64, 96


@pytest.fixture(scope="module", autouse=True)
def _built():
    mxbuild.build()


def good():
    u8, bf16 = dict(dtype=torch.uint8), dict(dtype=torch.bfloat16)
    return dict(x=torch.zeros((T, K), **bf16), logits=torch.zeros((T, E)), resid=torch.zeros((T, K), **bf16),
                w1=torch.zeros((E, 2, F, K // 2), **u8), s1=torch.zeros((E, 2, mx.mxfp4_scale_relayout_size(F, K)), **u8),
                w2=torch.zeros((E, K, F // 2), **u8), s2=torch.zeros((E, mx.mxfp4_scale_relayout_size(K, F)), **u8),
                w_pre=torch.zeros(K, **bf16), w_post=torch.zeros(K, **bf16), token_mask=torch.zeros(T, **u8))


def refusal(**changes):
    args = good()
    args.update({name: change(args[name]) for name, change in changes.items()})
    with pytest.raises((TypeError, ValueError)) as e:
        mx.moe_block(k=2, **args)
    return e.type, str(e.value)


def apart(t):
    """The same values with a gap after each element."""
    wide = torch.zeros((*t.shape, 2), dtype=t.dtype)
    wide[..., 0] = t
    return wide[..., 0]


def test_right_arguments_are_refused_for_their_place_alone():
    everything = (ValueError, "moe_block: everything on one GPU expected")
    assert refusal() == everything
    assert refusal(logits=lambda t: t.bfloat16(), token_mask=lambda t: t.bool()) == everything
    assert refusal(w_pre=lambda t: None, w_post=lambda t: None, token_mask=lambda t: None) == everything
    # Rows may be apart.
    assert refusal(x=lambda t: torch.zeros((T, K + 8), dtype=t.dtype)[:, :K], logits=lambda t: torch.zeros((T, 9))[:, 2:6]) == everything
    assert refusal(s1=lambda t: t.reshape(-1)) == everything
    # No tokens, whatever the strides of nothing.
    none = {name: lambda t: torch.empty_strided((0, t.shape[1]), (1, 7), dtype=t.dtype) for name in ("x", "logits", "resid")}
    none["token_mask"] = lambda t: t[:0]
    assert refusal(**none) == everything


@pytest.mark.parametrize("name,dtype", [("logits", torch.float16), ("logits", torch.float64), ("logits", torch.int32),
                                        ("x", torch.float16), ("x", torch.float32), ("resid", torch.float16),
                                        ("resid", torch.float32), ("w_pre", torch.float32), ("w_post", torch.float16),
                                        ("token_mask", torch.int32), ("token_mask", torch.float32), ("w1", torch.int32),
                                        ("w2", torch.bfloat16), ("s1", torch.float32), ("s2", torch.int16)])
def test_types(name, dtype):
    kind, text = refusal(**{name: lambda t: t.to(dtype)})
    assert kind is TypeError and name in text


@pytest.mark.parametrize("name", ["x", "logits", "resid", "w_pre", "w_post", "token_mask", "w1", "w2", "s1", "s2"])
def test_layouts(name):
    kind, text = refusal(**{name: apart})
    assert kind is ValueError and name in text


@pytest.mark.parametrize("name,cut", [("logits", lambda t: t[:, :3]), ("logits", lambda t: t[:9]), ("resid", lambda t: t[:9]),
                                      ("resid", lambda t: t[:, :32]), ("w_pre", lambda t: t[:63]), ("w_post", lambda t: t[:32]),
                                      ("token_mask", lambda t: t[:9]), ("w1", lambda t: t[:, :, :, :16]),
                                      ("w1", lambda t: t.transpose(1, 2)), ("w2", lambda t: t[:3]),
                                      ("w2", lambda t: t.transpose(1, 2)), ("s1", lambda t: t[:3]), ("s2", lambda t: t[..., 1:])])
def test_shapes(name, cut):
    kind, text = refusal(**{name: cut})
    assert kind is ValueError and (name in text or "w1" in text)


def test_relaid_expert_scales():
    S = torch.zeros((E, F, K // 32), dtype=torch.uint8)
    for bad, kind in ((S.int(), TypeError), (S[..., :1], ValueError), (S.reshape(-1), ValueError), (S, ValueError)):
        with pytest.raises(kind):
            mx.relaid_expert_scales(bad, K)
