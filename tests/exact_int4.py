"""4-bit integer linears and rows of x whose every product and sum is exact in fp32: x in -2..2, scales 1/2 and 1, a whole
bias. A result has to equal the rounding of the exact one, bit for bit."""

import numpy as np

from oracle import formats, int4 as oint4

CASES = [
    # T, N, K, group, zeros, type
    (1, 1, 128, 128, False, "bf16"), (1, 40, 32, 32, True, "f16"), (2, 50, 192, 64, True, "bf16"), (5, 33, 1056, 32, True, "f16"),
    (3, 1001, 1056, 32, True, "bf16"), (7, 2048, 2048, 128, False, "bf16"), (8, 12000, 1024, 32, True, "bf16"),
    (9, 250, 384, 64, True, "f16"), (16, 64, 2048, 128, False, "bf16"), (1, 6144, 6144, 128, True, "bf16"),
    (5, 4096, 6144, 64, True, "f16"), (40, 100, 640, 64, True, "bf16"),
    # K in parts: many units a CTA, an uneven last part, one row whose K does not fit, several passes
    (16, 12288, 6144, 128, False, "bf16"), (16, 40000, 4224, 128, True, "bf16"), (12, 3000, 6176, 32, True, "f16"),
    (1, 33, 131072, 128, True, "bf16"), (1, 33, 131072, 64, True, "f16"), (4, 33, 131072, 32, True, "bf16"), (16, 20, 32768, 128, True, "f16"),
    (33, 64, 9216, 64, True, "bf16"),
]


class ExactLinear:
    """codes, scales, zeros (or None), bias and x as numpy arrays; the numbers in float64."""

    def __init__(self, T, N, K, group, zeros, act, seed=0):
        r = np.random.default_rng(seed + N + K + T)
        self.group, self.act = group, act
        self.codes = r.integers(0, 256, (N, K // 2), dtype=np.uint8)
        self.scales = r.choice([0.5, 1.0], (N, K // group))
        self.zeros = r.integers(0, 16, (N, K // group), dtype=np.uint8) if zeros else None
        self.bias = r.integers(-8, 9, N).astype(np.float64)
        self.x = r.integers(-2, 3, (T, K)).astype(np.float64)
        self.w = oint4.weights(self.codes, self.scales, self.zeros, group)

    def result(self, lost=None):
        """out [T, N] rounded to the activation type; lost: a block of 128 of K left out."""
        x = self.x.astype(np.float32)
        w = self.w.astype(np.float32)
        assert (np.abs(x) @ np.abs(w).T).max() + 8 < 2 ** 23          # in units of a half below 2^24: exact
        if lost is not None:
            x[:, 128 * lost:128 * lost + 128] = 0
        return formats.act_rne((x @ w.T).astype(np.float64) + self.bias, self.act)
