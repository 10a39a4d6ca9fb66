"""A frozen 4-bit model with low-rank adapters: serving many requests, and training the router beside them.

  python examples/adapters.py        # needs a GB300 and the built library

1. serve:  a W4A16 projection, every request with its own adapter (or none).
2. expert: the hybrid MoE layer with a low-rank branch for each expert. The tokens are sorted by expert
           (ExpertRows.dispatch), the experts' adapters run on the sorted rows, and the gate-weighted sum
           (ExpertRows.combine) joins the frozen layer's output.
3. train:  the gradient of that branch with respect to its rows, the gates and the router's logits.
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import nf3_moe_gb300 as hm  # noqa: E402
import synth  # noqa: E402


def serve(tokens=24, requests=6, K=512, N=384, rank=16):
    """y = W x + scale_a B_a A_a x with a of each token's request; returns what the caller may check."""
    torch.manual_seed(0)
    w = 0.02 * torch.randn((N, K), device="cuda")
    codes, scales, g = synth.quant_nvfp4(w)
    linear = hm.LinearW4A16(N, K, hm.FMT_NVFP4, codes, scales, g, max_tokens=tokens)
    adapters = hm.LoraAdapters(K, N, slots=requests, max_rank=rank, max_tokens=tokens)
    weights = {}
    for a in range(requests - 1):                                   # the last request has no adapter
        r = 1 + (5 * a) % rank
        A = (torch.randn((r, K), device="cuda") * K ** -0.5).bfloat16()
        B = (torch.randn((N, r), device="cuda") * 0.1).bfloat16()
        adapters.load(a, A, B, scale=2.0)
        weights[a] = (A, B, 2.0)
    x = synth.gen_x(tokens, K, device="cuda")
    ids = torch.arange(tokens, device="cuda", dtype=torch.int32) * requests // tokens   # a request's tokens side by side
    ids = torch.where(ids == requests - 1, torch.full_like(ids, -1), ids)
    y = linear(x, adapters=adapters, ids=ids)
    hm.hmoe_check_device_status(adapters.ws)
    return x, ids, weights, linear(x), y


class ExpertBranch:
    """A low-rank branch for every expert of a HybridMoELayer, beside the frozen layer."""

    def __init__(self, moe, rank, max_tokens):
        H, E, k = moe.H, moe.E, moe.topk
        self.moe = moe
        self.rows_of = hm.ExpertRows(H, E, k, max_tokens=max_tokens, dtype=moe.dtype)
        self.adapters = hm.LoraAdapters(H, H, slots=E, max_rank=rank, max_tokens=max_tokens * k)

    def branch(self, x, logits, routes):
        """sum_j gate_j * scale B_e A_e x over the token's experts; the sorted rows and their results too."""
        ids, gates, perm, offsets = routes
        rows, plan = self.rows_of.dispatch(x, perm, offsets)
        expert_of_row = ids.reshape(-1)[plan.row_slot.long()]      # no padding here (align=1): every row has a slot
        z = self.adapters(rows.detach(), expert_of_row)            # they have no gradient: constants up to here
        z.requires_grad_(logits.requires_grad)
        return self.rows_of.combine(z, plan, gates, ids=ids, logits=logits), z, plan

    def __call__(self, x, logits):
        routes = self.moe.plan(logits.detach())
        ids, gates, perm, offsets = routes
        out = torch.empty((x.shape[0], self.moe.H), dtype=self.moe.dtype, device=x.device)
        hm.hmoe_forward(self.moe.layer, x, ids, gates, perm, offsets, out, self.moe.ws)
        delta, z, plan = self.branch(x, logits, routes)
        return out + delta, out, z, plan, routes


def expert_branch(tokens=40, rank=8):
    torch.manual_seed(1)
    L = synth.tiny_layer(device="cuda")
    experts = [(e["w13"][0], e["w13"][1], e["w13"][2], e["w2"][0], e["w2"][1], e["w2"][2]) for e in L.experts]
    moe = hm.HybridMoELayer(L.H, L.I, L.E, L.topk, [int(b) for b in L.bit_map], experts, max_tokens=tokens)
    net = ExpertBranch(moe, rank, tokens)
    weights = []
    for e in range(L.E):
        A = (torch.randn((rank, L.H), device="cuda") * L.H ** -0.5).bfloat16()
        B = (torch.randn((L.H, rank), device="cuda") * 0.1).bfloat16()
        net.adapters.load(e, A, B, scale=1.0)
        weights.append((A, B))
    x = synth.gen_x(tokens, L.H, device="cuda")
    logits = synth.gen_logits(tokens, L.E, device="cuda").requires_grad_()
    y, frozen, z, plan, routes = net(x, logits)
    dy = torch.randn_like(y)
    y.backward(dy)                                                 # z.grad and logits.grad
    for ws in (moe.ws, net.rows_of.ws, net.adapters.ws):
        hm.hmoe_check_device_status(ws)
    return dict(x=x, logits=logits, y=y, frozen=frozen, z=z, plan=plan, routes=routes, dy=dy, weights=weights)


def main():
    x, ids, weights, plain, y = serve()
    print(f"serve: {x.shape[0]} tokens, {len(weights)} adapters, |change| of the projection up to {float((y - plain).abs().max()):.3f}")
    r = expert_branch()
    print(f"expert branch: {r['x'].shape[0]} tokens as {r['z'].shape[0]} rows, "
          f"|branch| up to {float((r['y'] - r['frozen']).detach().abs().max()):.3f}, |d logits| up to {float(r['logits'].grad.abs().max()):.3f}")


if __name__ == "__main__":
    main()
