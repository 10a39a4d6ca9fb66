"""Layers and tokens whose every product and sum is exact in fp32, so that a kernel's result has to equal the rounding of
the exact one, bit for bit. For the tests of the whole layer for a few tokens, on the CPU and the GPU.

Weights are -1, 0 and 1, x is a token's a or 2a. A gate row has a one in every 64 of K, so that silu's argument is at
least 18 (there silu(z) = z in fp32) and lacks something where any k-block is left out; an up row has up to eight of
-1 and 1, a row of W2 one of them in every 64 of I, and four at least, times 2^-8. h = z u is a whole number below 2^15, with more digits than one
value of the activation type holds. The router gives a token's k experts the same logit: their gates are 1 / k, k a power
of two. Sums stay below 2^24 of their unit (asserted)."""

import numpy as np
import torch

import synth
from oracle import formats

SHIFT = 8      # of W2
MARKS = 16     # values of K, of which no weight is: value t marks token t


def encode(fmt, w, shift, device):
    """codes, scales and the global scale of w in -1, 0, 1 times 2^-shift."""
    N, K = w.shape
    w = torch.from_numpy(w)
    if fmt == synth.FMT_NF3:
        code = torch.where(w == 0, 3, torch.where(w > 0, 7, 0))
        scale = torch.full((N, K // 64), 2.0 ** -shift, dtype=torch.bfloat16).view(torch.int16)
        return synth.pack_nf3_bits(code).to(device), scale.to(device), 1.0
    code = (torch.where(w == 0, 0, 2) | torch.where(w < 0, 8, 0)).to(torch.uint8)
    codes = (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous().to(device)
    if fmt == synth.FMT_NVFP4:
        return codes, torch.full((N, K // 16), 0x38, dtype=torch.uint8, device=device), 2.0 ** -shift  # E4M3 one
    return codes, torch.full((N, K // 32), 127 - shift, dtype=torch.uint8, device=device), 1.0


class ExactLayer:
    """layer: a synth.Layer; x [T, H] and router [E, H], whole numbers in float64; ids [T, k]; w13, w2: the whole weights."""

    def __init__(self, T, H, I, E, k, kept_format, kept, act, device="cpu", seed=0):
        assert k & (k - 1) == 0 and T <= MARKS
        r = np.random.default_rng(seed + 7 * H + I)
        self.T, self.H, self.I, self.k, self.act = T, H, I, k, act
        nb, nb2 = H // 64, I // 64
        a = -(-18 // nb)
        self.x = a * r.integers(1, 3, (T, H)).astype(np.float64)
        self.x[:, :MARKS] = 0
        self.x[np.arange(T), np.arange(T)] = 1
        self.ids = np.stack([np.sort(r.permutation(E)[:k]) for _ in range(T)])
        self.router = np.zeros((E, H))
        for t in range(T):
            self.router[self.ids[t], t] = 64
        bit_map = None if kept is None else np.full(E, 3, dtype=np.int8)
        if kept is not None:
            bit_map[r.permutation(E)[:kept]] = 4
        self.w13, self.w2, experts = {}, {}, []
        for e in range(E):
            fmt = kept_format if bit_map is None or bit_map[e] == 4 else synth.FMT_NF3
            w = np.zeros((2 * I, H), dtype=np.int8)
            rows = np.arange(I)
            for b in range(nb):
                w[rows, 64 * b + r.integers(MARKS, 64, I)] = 1
            for _ in range(min(8, nb)):
                w[I + rows, 64 * r.integers(0, nb, I) + r.integers(MARKS, 64, I)] = r.choice([-1, 1], I)
            v = np.zeros((H, I), dtype=np.int8)
            for b in range(max(nb2, 4)):
                v[np.arange(H), 64 * (b % nb2) + r.integers(0, 64, H)] = r.choice([-1, 1], H)
            used = (self.ids == e).any()
            if used:
                self.w13[e], self.w2[e] = w, v
            experts.append({"fmt": fmt, "w13": encode(fmt, w, 0, device), "w2": encode(fmt, v, SHIFT, device)})
        self.layer = synth.Layer(H, I, E, k, bit_map, kept_format, experts, act)

    def result(self, drop_slot=False, drop13=None, drop2=None, h_of=None):
        """out [T, H] rounded to the activation type. Mistakes on demand: a token's last slot, a k-block of W13 or of W2
        left out, h through a function."""
        out = np.zeros((self.T, self.H))
        size = np.zeros((self.T, self.H))
        for e, w in self.w13.items():
            x = self.x.copy()
            if drop13 is not None:
                x[:, 64 * drop13:64 * drop13 + 64] = 0
            rows = np.flatnonzero((self.ids[:, :-1] == e).any(axis=1) if drop_slot else (self.ids == e).any(axis=1))
            if len(rows) == 0:
                continue
            gu = x[rows].astype(np.float32) @ w.astype(np.float32).T  # whole numbers below 2^24: exact
            z, u = gu[:, :self.I], gu[:, self.I:]
            if drop13 is None:
                assert z.min() >= 18 and np.abs(z * u).max() < 2 ** 15
            h = z * u
            h = h if h_of is None else h_of(h)
            if drop2 is not None:
                h[:, 64 * drop2:64 * drop2 + 64] = 0
            v = self.w2[e].astype(np.float32).T
            h = h.astype(np.float32)
            out[rows] += h @ v
            size[rows] += np.abs(h) @ np.abs(v)
        assert size.max() * self.k < 2 ** 24
        return formats.act_rne(out / self.k * 2.0 ** -SHIFT, self.act)


CASES = [
    # T, H, I, E, k, kept format, kept experts (None: no bit map), type
    (1, 128, 64, 1, 1, synth.FMT_NVFP4, None, "bf16"),
    (8, 128, 64, 8, 8, synth.FMT_NVFP4, None, "bf16"),            # every token to every expert
    (8, 256, 128, 8, 2, synth.FMT_NVFP4, 4, "bf16"),
    (5, 256, 192, 6, 4, synth.FMT_MXFP4, 3, "f16"),               # odd k-blocks of W2
    (8, 384, 320, 16, 4, synth.FMT_NVFP4, 5, "bf16"),
    (3, 256, 128, 40, 32, synth.FMT_NVFP4, 20, "bf16"),           # the largest top-k
    (8, 128, 64, 40, 32, synth.FMT_MXFP4, 20, "f16"),
    (7, 128, 704, 3, 2, synth.FMT_NVFP4, 0, "f16"),               # nothing kept
    (2, 2048, 768, 24, 8, synth.FMT_NVFP4, None, "bf16"),
    (6, 1024, 512, 5, 1, synth.FMT_MXFP4, 2, "bf16"),
    (8, 8192, 64, 2, 1, synth.FMT_NVFP4, 1, "bf16"),              # activations that fit a few tokens at a time
    (6, 128, 4096, 2, 2, synth.FMT_NVFP4, 1, "f16"),
    # with 16 warps
    (8, 1024, 704, 40, 8, synth.FMT_NVFP4, 20, "bf16"),
    (8, 640, 832, 16, 16, synth.FMT_MXFP4, 6, "f16"),             # every token to every expert, odd k-blocks of W2
    (1, 4096, 1216, 8, 8, synth.FMT_NVFP4, 4, "bf16"),
    (4, 6144, 2048, 8, 4, synth.FMT_NVFP4, 3, "bf16"),
    (8, 8192, 256, 16, 4, synth.FMT_NVFP4, 8, "f16"),
    (6, 128, 9792, 8, 8, synth.FMT_NVFP4, 3, "bf16"),
    # the limits: activations of one token fill shared memory
    (3, 39680, 64, 2, 1, synth.FMT_NVFP4, 1, "bf16"),
    (3, 128, 19840, 2, 2, synth.FMT_MXFP4, 1, "f16"),
    (8, 39680, 320, 4, 2, synth.FMT_NVFP4, 2, "f16"),             # with 16 warps
]
