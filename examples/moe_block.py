"""A mixture-of-experts layer on MXFP4 weights, from the residual stream back to it.

    python examples/moe_block.py [--tokens T] [--steps N]

Expert weights are quantised once with mxfp4_quantize and their scales laid out
once.  Then a prompt's tokens go through the layer in one pass (some of them
padding), and single tokens as a decoding loop sends them, replayed from a CUDA
graph.  The prompt's result is compared with the same layer in fp32 on
dequantised operands.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_mxfp4_gb300 as mx

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def quantised(w):
    """bf16 [..., N, K] -> packed codes [..., N, K / 2], scales [..., N, K / 32]."""
    rows, K = w.numel() // w.shape[-1], w.shape[-1]
    q = torch.empty((*w.shape[:-1], K // 2), dtype=torch.uint8, device=w.device)
    s = torch.empty((*w.shape[:-1], K // 32), dtype=torch.uint8, device=w.device)
    mx.mxfp4_quantize(q, K, s, K // 32, w, K, rows, K)
    return q, s


def dequantised(q, s):
    table = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=q.device)
    v = torch.stack([table[(q & 15).long()], table[(q >> 4).long()]], -1).flatten(-2)
    return v * torch.exp2(s.float() - 127).repeat_interleave(32, -1)


def norm(x, w, eps=1e-6):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w


class Layer:
    def __init__(self, experts, k, hidden, inner):
        rand = lambda *shape: torch.randn(shape, device="cuda") * shape[-1] ** -0.5
        self.k, self.router = k, rand(experts, hidden)
        self.w1, self.s1 = quantised(rand(experts, 2, inner, hidden).bfloat16())
        self.w2, self.s2 = quantised(rand(experts, hidden, inner).bfloat16())
        self.r1 = mx.relaid_expert_scales(self.s1, hidden)
        self.r2 = mx.relaid_expert_scales(self.s2, inner)
        self.w_next = (1 + 0.1 * torch.randn(hidden, device="cuda")).bfloat16()

    def __call__(self, normed, resid, mask=None):
        """(The residual stream after the layer, its norm for the next one.)"""
        logits = normed.float() @ self.router.T
        return mx.moe_block(normed, logits, resid, self.w1, self.r1, self.w2, self.r2, self.k,
                            w_pre=self.w_next, token_mask=mask)

    def plain(self, normed, resid, mask):
        v, ids = (normed.float() @ self.router.T).topk(self.k)
        x = dequantised(*quantised(normed))
        gates = v.softmax(-1) * mask[:, None]
        out = resid.float()
        for e in range(self.router.shape[0]):
            g = (gates * (ids == e)).sum(-1, keepdim=True)
            gate, up = dequantised(self.w1[e], self.s1[e])
            h = torch.nn.functional.silu(x @ gate.T) * (x @ up.T)
            h = dequantised(*quantised(h.bfloat16()))
            out = out + g * (h @ dequantised(self.w2[e], self.s2[e]).T)
        return out, norm(out, self.w_next.float())


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--experts", type=int, default=32)
    ap.add_argument("--topk", type=int, default=4)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--inner", type=int, default=1024)
    a = ap.parse_args()
    torch.manual_seed(0)
    layer = Layer(a.experts, a.topk, a.hidden, a.inner)

    resid = torch.randn((a.tokens, a.hidden), device="cuda").bfloat16()
    normed = norm(resid.float(), torch.ones(a.hidden, device="cuda")).bfloat16()
    mask = torch.ones(a.tokens, dtype=torch.uint8, device="cuda")
    mask[a.tokens - a.tokens // 8:] = 0                 # padding: no expert, the residual passes
    h, n = layer(normed, resid, mask)
    want_h, want_n = layer.plain(normed, resid, mask)
    part = lambda got, want: ((got.float() - want).norm() / want.norm()).item()
    layer_part = ((h.float() - want_h).norm() / (want_h - resid.float()).norm()).item()
    print(f"prompt of {a.tokens}: relative difference {part(h, want_h):.4f} of the stream, "
          f"{part(n, want_n):.4f} of its norm, {layer_part:.3f} of the layer's own part")
    assert torch.equal(h[mask == 0], resid[mask == 0])
    # The plain form rounds the hidden values to bf16 before it quantises them, so
    # some of their FP4 codes differ by a step.
    assert layer_part < 0.1

    x1, r1 = normed[:1].clone(), resid[:1].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(x1, r1)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h1, n1 = layer(x1, r1)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(a.steps):
        graph.replay()
        r1.copy_(h1)                                    # as the next layer of the same token
        x1.copy_(n1)
    end.record()
    torch.cuda.synchronize()
    assert mx.mxfp4_device_status() == 0 and torch.isfinite(h1).all()
    print(f"{a.steps} steps of one token: {start.elapsed_time(end) / a.steps * 1e3:.1f} us each")


if __name__ == "__main__":
    main()
