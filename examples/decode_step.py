"""A decode step with 4-bit weights throughout: an integer projection, the hybrid MoE layer from hidden states, the
logits of an integer head, captured once in a CUDA graph and replayed for every step.

  python examples/decode_step.py        # needs a GB300 and the built library
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import nf3_moe_gb300 as hm  # noqa: E402
import synth  # noqa: E402


def quant_int4(w, group):
    """codes, scales and zero points of weights [N, K]: each group's range in 16 even steps."""
    N, K = w.shape
    g = w.view(N, K // group, group)
    lo, hi = g.amin(dim=2).clamp(max=0), g.amax(dim=2).clamp(min=0)
    scale = ((hi - lo) / 15).bfloat16()
    zero = torch.round(-lo / scale.float()).clamp(0, 15)
    q = torch.round(g / scale.float()[:, :, None] + zero[:, :, None]).clamp(0, 15).to(torch.uint8).view(N, K)
    return q[:, 0::2] | (q[:, 1::2] << 4), scale, zero.to(torch.uint8)


class Block:
    """z = x + W x;  h = z + moe(z);  logits = V h."""

    def __init__(self, tokens, vocabulary=1000, group=64):
        torch.manual_seed(0)
        self.L = synth.tiny_layer(device="cuda")
        H = self.L.H
        experts = [(*e["w13"], *e["w2"]) for e in self.L.experts]
        self.moe = hm.HybridMoELayer(H, self.L.I, self.L.E, self.L.topk, [int(b) for b in self.L.bit_map], experts, max_tokens=tokens)
        self.router = (torch.randn((self.L.E, H), device="cuda") * H ** -0.5).bfloat16()
        self.bias = 0.1 * torch.randn(self.L.E, device="cuda")
        self.packed = {}
        for name, n in (("proj", H), ("head", vocabulary)):
            self.packed[name] = quant_int4(torch.randn((n, H), device="cuda") * H ** -0.5, group)
        self.proj = hm.LinearInt4(H, H, group, *self.packed["proj"])
        self.head = hm.LinearInt4(vocabulary, H, group, *self.packed["head"])

    def __call__(self, x):
        y = self.proj(x)
        z = x + y
        m, ids, gates = self.moe.decode(z, self.router, bias=self.bias)
        h = z + m
        return dict(y=y, z=z, m=m, ids=ids, gates=gates, h=h, logits=self.head(h))


def graph_of(block, x):
    """The step on the static input x as a graph, and its outputs."""
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        block(x)                                                   # once outside the capture
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out = block(x)
    torch.cuda.current_stream().wait_stream(stream)
    return graph, out


def main(tokens=4, steps=8):
    block = Block(tokens)
    x = synth.gen_x(tokens, block.L.H, device="cuda")
    graph, out = graph_of(block, x)
    for step in range(steps):
        graph.replay()
        chosen = out["logits"].float().argmax(dim=1)
        print(f"step {step}: tokens {chosen.tolist()}, experts of the first {out['ids'][0].tolist()}")
        x.copy_(synth.gen_x(tokens, block.L.H, seed=step + 1, device="cuda"))   # the next tokens' hidden states
    hm.hmoe_check_device_status(block.moe.decode_ws)


if __name__ == "__main__":
    main()
