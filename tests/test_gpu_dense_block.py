"""The dense layer and its gradients as they run together, against the 64-bit forms
of tests/dense_block_ref.py."""
import os
import subprocess
import sys

import numpy as np
import pytest

import block_scaled_mxfp4_gb300 as mx
import dense_block_ref as br
import dense_ref as dr
import expert_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

FMT = {"e4m3": mx.MXFP8_E4M3, "e5m2": mx.MXFP8_E5M2}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from block_scaled_mxfp4_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    mx.mxfp4_device_status(reset=True)
    yield
    assert mx.mxfp4_device_status() == 0, "a bounded wait timed out during the tests"


def host(t):
    torch.cuda.synchronize()
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


class Layer:
    """Weights, inputs and their 64-bit values."""

    def __init__(self, T, K, F, fmt="e4m3", act="gelu", bias="bf16", norm="fp32", seed=0, apart=0):
        rng = np.random.default_rng(seed + T + K + F)
        self.T, self.K, self.F, self.fmt, self.act = T, K, F, fmt, act
        types = {"bf16": torch.bfloat16, "fp32": torch.float32}

        def made(v, kind="bf16"):
            return None if kind is None else torch.from_numpy(v).to(types[kind]).cuda()

        flat = made(rng.normal(size=(T, K + apart)) * np.exp(rng.normal(size=(T, 1))) + 0.3)
        self.x = flat[:, :K]
        self.dout = made(rng.normal(size=(T, K)))
        w1, w2 = made(rng.normal(size=(F, K)) * K ** -0.5), made(rng.normal(size=(K, F)) * F ** -0.5)
        self.b1, self.b2 = made(rng.normal(size=F) * 0.3, bias), made(rng.normal(size=K) * 0.3, bias)
        self.nw, self.nb = made(1 + 0.2 * rng.normal(size=K), norm), made(0.1 * rng.normal(size=K), norm)
        self.plain = {"w1": host(w1), "w2": host(w2)}
        if fmt == "e2m1":
            self.w = []
            for w in (w1, w2):
                q, s = (torch.empty((w.shape[0], w.shape[1] // n), dtype=torch.uint8, device="cuda") for n in (2, 32))
                mx.mxfp4_quantize(q, w.shape[1], s, w.shape[1] // 32, w, w.shape[1], *w.shape)
                self.w += [q, s]
        else:
            self.f1, self.f2 = (mx.mxfp8_forms(w, FMT[fmt]) for w in (w1, w2))
            self.w = [self.f1.q, self.f1.s, self.f2.q, self.f2.s]
        value = lambda q, s: ref.values(host(q), host(s), fmt)
        zero = lambda t, v: v if t is None else host(t)
        self.p = dict(x=host(self.x), w1=value(*self.w[:2]), w2=value(*self.w[2:]), b1=zero(self.b1, 0.0), b2=zero(self.b2, 0.0),
                      norm_w=zero(self.nw, np.ones(K)), norm_b=zero(self.nb, np.zeros(K)), act=act, eps=1e-5)
        if fmt != "e2m1":
            self.p.update(w1t=value(self.f1.qt, self.f1.st)[:, :F], w2t=value(self.f2.qt, self.f2.st)[:, :K])

    def __call__(self, keep=False, stream=None, x=None):
        return mx.dense_block(self.x if x is None else x, *self.w, self.b1, self.b2, self.nw, self.nb, dr.ACTS.index(self.act),
                              FMT.get(self.fmt, 0), 1e-5, keep, stream)

    def grads(self, kept, fmt_grad="e4m3", stream=None, dout=None):
        return mx.dense_block_backward(self.dout if dout is None else dout, kept, self.f1.qt, self.f1.st, self.f2.qt, self.f2.st,
                                       FMT[fmt_grad], stream)


def within(got, want, what, slack=0.0):
    v, e = want
    bad = ~(np.abs(got - v) <= e * (1 + 1e-9) + slack)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}; {got[bad][:3]} for {v[bad][:3]} within {np.broadcast_to(e, v.shape)[bad][:3]}"


SHAPES = [(1, 32, 32), (3, 64, 96), (37, 96, 160), (130, 320, 1280), (257, 544, 288), (2309, 512, 2304)]


@pytest.mark.parametrize("T,K,F", SHAPES)
@pytest.mark.parametrize("fmt,act", [("e2m1", "gelu_tanh"), ("e4m3", "silu"), ("e5m2", "relu")])
def test_forward(T, K, F, fmt, act):
    p = Layer(T, K, F, fmt, act, bias="fp32" if fmt == "e2m1" else "bf16", apart=5)
    out = p()
    want = br.forward(p.p, br.Rounded, fmt)
    within(host(out), want["out"], "out")
    assert out.shape == (T, K)
    # Only values beside a rounding's edge are open: y's bound, about 2^-17 of it, over a step of
    # 2^-8 of it on either side is some 3 in a thousand (of a few hundred values, one or several).
    assert (want["y"][1] > 0).mean() < 1e-2 or T * K < 10_000


@pytest.mark.parametrize("T,K,F", SHAPES)
@pytest.mark.parametrize("act", dr.ACTS)
def test_gradients(T, K, F, act):
    fmt, fmt_grad = ("e4m3", "e5m2") if act == "silu" else ("e5m2", "e4m3") if act == "relu" else ("e4m3", "e4m3")
    p = Layer(T, K, F, fmt, act, bias=None if act == "none" else "bf16", norm="bf16" if act == "none" else "fp32")
    out, kept = p(keep=True)
    assert torch.equal(out, p())
    want = br.forward(p.p, br.Rounded, fmt)
    within(host(out), want["out"], "out")
    mean, rstd = host(kept.mean), host(kept.rstd)
    within(mean, (want["mean"], want["emean"]), "mean")
    within(rstd, (want["rstd"], want["erstd"]), "rstd")
    dr.check_codes(host(kept.z), host(kept.sz), *want["z"], fmt, "z")
    dr.check_codes(host(kept.yt), host(kept.syt), np.ascontiguousarray(want["y"][0].T), np.ascontiguousarray(want["y"][1].T), fmt, "y^T")
    z = ref.values(host(kept.z), host(kept.sz), fmt)
    yt = ref.values(host(kept.yt), host(kept.syt), fmt)[:, :T]
    g = p.grads(kept, fmt_grad)
    wants = br.backward(dict(p.p, mean=mean, rstd=rstd), host(p.dout), (yt, np.zeros_like(yt)), (z, np.zeros_like(z)), br.Rounded, fmt,
                        fmt_grad)
    for name, got in g._asdict().items():
        within(host(got), wants[name], name)


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu", "none"])
def test_gradients_against_differences(act):
    """The formulas in real numbers against central differences of the layer's definition, and the
    kernels' gradients within their roundings of them."""
    T, K, F = 5, 64, 32
    p = Layer(T, K, F, "e4m3", act, norm="fp32")
    dout = host(p.dout)
    w1, w2 = p.plain["w1"], p.plain["w2"]
    real = dict(p.p, w1=w1, w2=w2, w1t=w1.T.copy(), w2t=w2.T.copy())
    names = {"dx": "x", "dw1": "w1", "dw2": "w2", "db1": "b1", "db2": "b2", "dnorm_w": "norm_w", "dnorm_b": "norm_b"}

    def loss(**changes):
        q = dict(real, **changes)
        y = dr.norm(q["x"], q["norm_w"], q["norm_b"], q["eps"])[0]
        return ((dr.act(y @ q["w1"].T + q["b1"], act)[0] @ q["w2"].T + q["b2"] + q["x"]) * dout).sum()

    y, mean, rstd, ey, em, er = dr.norm(real["x"], real["norm_w"], real["norm_b"], real["eps"])
    codes = lambda v: br.Loose.codes(v, np.zeros_like(v), "e4m3")
    real["ew1t"], real["ew2t"] = codes(real["w1t"])[1], codes(real["w2t"])[1]
    ybf = br.Loose.bf16(y, ey)
    z = br.matmul(*br.Loose.codes(*ybf, "e4m3"), w1, codes(w1)[1])
    z = br.Loose.codes(z[0] + real["b1"], z[1] + 1e-6, "e4m3")
    # Statistics in fp32 move the norm's gradients by less than 2^-16 of their terms; the bounds of
    # the 8-bit roundings, 2^-4 and more of them, are taken a hundredth larger for it.
    wants = br.backward(dict(real, mean=mean, rstd=rstd), dout, br.Loose.codes(ybf[0].T.copy(), ybf[1].T.copy(), "e4m3"), z, br.Loose,
                        "e4m3", "e4m3")
    out, kept = p(keep=True)
    g = p.grads(kept)
    n = 1e-5
    rng = np.random.default_rng(0)
    for name, of in names.items():
        v, e = wants[name]
        got = host(getattr(g, name))
        within(got, (v, 1.01 * e), name, slack=1e-6)
        base = real[of]
        for _ in range(40):
            at = tuple(rng.integers(0, m) for m in base.shape)
            step = np.zeros_like(base)
            step[at] = n
            diff = (loss(**{of: base + step}) - loss(**{of: base - step})) / (2 * n)
            assert abs(diff - v[at]) <= 1e-6 * (1 + abs(diff)), (name, at, diff, v[at])


def test_no_tokens():
    p = Layer(4, 64, 96)
    out, kept = p(keep=True, x=p.x[:0])
    g = p.grads(kept, dout=p.dout[:0])
    assert out.shape == (0, 64) and g.dx.shape == (0, 64)
    torch.cuda.synchronize()
    assert all((t == 0).all() for t in g)


def test_a_lone_row_of_any_stride():
    p = Layer(1, 96, 160)
    lone = lambda t: t.reshape(-1)[:, None].t()
    assert lone(p.x).stride(0) == 1
    out, kept = p(keep=True)
    o2, k2 = p(keep=True, x=lone(p.x))
    g, g2 = p.grads(kept), p.grads(k2, dout=lone(p.dout))
    torch.cuda.synchronize()
    assert torch.equal(out, o2) and all(torch.equal(a, b) for a, b in zip(g, g2))


def test_another_stream_and_two_graphs():
    """The layer and its gradients on a stream of their own, and captured for two inputs, replayed in
    turn with an eager pass of the same weights between them."""
    p = Layer(200, 320, 640)
    want = p(keep=True)
    wants = [want[0], *p.grads(want[1])]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, kept = p(keep=True, stream=s)
    got = [out, *p.grads(kept, stream=s.cuda_stream)]
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, wants))
    graphs = []
    for _ in range(2):
        x, dout = p.x.clone(), p.dout.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out, kept = p(keep=True, x=x)
            outs = [out, *p.grads(kept, dout=dout)]
        graphs.append((g, x, dout, outs))
    for _ in range(3):
        for g, x, dout, outs in graphs:
            x.normal_()
            dout.normal_()
            g.replay()
        for g, x, dout, outs in graphs:
            out, kept = p(keep=True, x=x)
            now = [out, *p.grads(kept, dout=dout)]
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(now, outs))


def test_calls_back_to_back_repeat():
    """Memory that one call gives back and the next one gets: the same bits each time."""
    p = Layer(700, 512, 1024, act="gelu")
    out, kept = p(keep=True)
    first = [out, *p.grads(kept)]
    for _ in range(5):
        out, kept = p(keep=True)
        again = [out, *p.grads(kept)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_is_not_finite_stays_in_its_row(bad):
    p = Layer(70, 96, 160)
    want = p()
    x = p.x.clone()
    x[13, 5] = bad
    got = p(x=x)
    torch.cuda.synchronize()
    rows = torch.arange(70, device="cuda") != 13
    assert got[13].isnan().all() and torch.equal(got[rows], want[rows])


def test_example():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, os.path.join(root, "examples", "dense_block.py"), "--tokens", "96", "--hidden", "64", "--inner",
                          "128", "--steps", "3"], capture_output=True, text=True, timeout=600)
    assert run.returncode == 0, run.stdout + run.stderr
