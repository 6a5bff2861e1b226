"""A transformer's dense layer on block-scaled weights: trained in MXFP8, served in MXFP4.

    python examples/dense_block.py [--tokens T] [--steps N]

Master weights are fp32; each step quantises them once in both orientations, runs the
layer and its gradients and moves the weights by plain gradient descent towards a layer
with other weights.  The first step's gradients are compared with the same layer in fp32.
Then the weights are quantised to MXFP4 and single tokens go through the layer, replayed
from a CUDA graph.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_mxfp4_gb300 as mx


class Layer:
    def __init__(self, hidden, inner, act=mx.MXFP4_ACT_GELU):
        rand = lambda *shape: torch.randn(shape, device="cuda") * shape[-1] ** -0.5
        self.act = act
        self.w1, self.w2 = rand(inner, hidden), rand(hidden, inner)
        self.b1, self.b2 = torch.zeros(inner, device="cuda"), torch.zeros(hidden, device="cuda")
        self.norm_w, self.norm_b = torch.ones(hidden, device="cuda"), torch.zeros(hidden, device="cuda")

    def weights(self):
        return [self.w1, self.w2, self.b1, self.b2, self.norm_w, self.norm_b]

    def plain(self, x):
        y = torch.nn.functional.layer_norm(x, x.shape[-1:], self.norm_w, self.norm_b)
        return x + torch.nn.functional.gelu(y @ self.w1.T + self.b1) @ self.w2.T + self.b2

    def step(self, x, gradient_of):
        """(out, gradients) of one pass; gradient_of(out) is the loss's gradient."""
        f1, f2 = mx.mxfp8_forms(self.w1.bfloat16()), mx.mxfp8_forms(self.w2.bfloat16())
        out, kept = mx.dense_block(x, f1.q, f1.s, f2.q, f2.s, self.b1, self.b2, self.norm_w, self.norm_b,
                                   self.act, keep=True)
        return out, mx.dense_block_backward(gradient_of(out), kept, f1.qt, f1.st, f2.qt, f2.st)

    def served(self):
        """The layer on MXFP4 weights: a function of the tokens."""
        def quantised(w):
            q, s = (torch.empty((w.shape[0], w.shape[1] // n), dtype=torch.uint8, device="cuda") for n in (2, 32))
            mx.mxfp4_quantize(q, w.shape[1], s, w.shape[1] // 32, w, w.shape[1], *w.shape)
            return q, s
        w1, w2 = quantised(self.w1.bfloat16()), quantised(self.w2.bfloat16())
        return lambda x: mx.dense_block(x, *w1, *w2, self.b1, self.b2, self.norm_w, self.norm_b, self.act)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--inner", type=int, default=8192)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--rate", type=float, default=4.0, help="over the inner size, which the loss's curvature grows with")
    a = ap.parse_args()
    torch.manual_seed(0)
    torch.backends.cuda.matmul.allow_tf32 = False
    layer, aim = Layer(a.hidden, a.inner), Layer(a.hidden, a.inner)
    x = torch.randn((a.tokens, a.hidden), device="cuda").bfloat16()
    target = aim.plain(x.float())

    for n in range(a.steps):
        loss = None

        def gradient_of(out):
            nonlocal loss
            off = out.float() - target
            loss = (off * off).mean()
            return (2 * off / a.tokens).bfloat16()

        out, g = layer.step(x, gradient_of)
        if n == 0:
            leaves = [t.requires_grad_() for t in layer.weights()]
            ((layer.plain(x.float()) - target) ** 2).sum().div(a.tokens).backward()
            for name, t, got in zip(("w1", "w2", "b1", "b2", "norm_w", "norm_b"), leaves,
                                    (g.dw1, g.dw2, g.db1, g.db2, g.dnorm_w, g.dnorm_b)):
                part = ((got.float() - t.grad).norm() / t.grad.norm()).item()
                print(f"gradient of {name}: relative difference {part:.4f} from fp32")
                # An E4M3 code is within 2^-4 of its value, an eighth at the scale's end; a few
                # of these lie behind each gradient.
                assert part < 0.25
                t.requires_grad_(False)
        for t, d in zip(layer.weights(), (g.dw1, g.dw2, g.db1, g.db2, g.dnorm_w, g.dnorm_b)):
            t -= a.rate / a.inner * d.float()
        if n % 5 == 0 or n == a.steps - 1:
            print(f"step {n}: loss {loss.item():.4f}")

    serve = layer.served()
    x1 = x[:1].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        serve(x1)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out1 = serve(x1)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(100):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    assert mx.mxfp4_device_status() == 0 and torch.isfinite(out1).all()
    print(f"one token through the MXFP4 layer: {start.elapsed_time(end) * 10:.1f} us")


if __name__ == "__main__":
    main()
