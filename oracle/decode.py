"""Oracle of the whole layer for a few tokens: router logits, top-k, gates, experts, sum. Float64 NumPy.

TEST INFRASTRUCTURE ONLY: see the package docstring.

No page defines the entry point; the parts are the layer's. The weights are the formats' values without a
rounding to the activation type (NF3: codebook entry times scale, exactly), and h is not rounded.
"""

import numpy as np

from . import formats, route


def weights(fmt, codes, scales, g, K):
    """[N, K] of one matrix in a logical layout of oracle.formats, NF3 unrounded."""
    if fmt != formats.FMT_NF3:
        return formats.dequant(fmt, codes, scales, g, K)
    value = formats.nf3_codebook()[formats.unpack_nf3(codes, K)]
    return value * np.repeat(formats.bf16_bits_to_f64(scales), formats.NF3_GROUP, axis=1)


def logits(x, router, bias=None):
    l = np.asarray(x, dtype=np.float64) @ np.asarray(router, dtype=np.float64).T
    return l if bias is None else l + np.asarray(bias, dtype=np.float64)


def choose(l, k):
    """ids [T, k] and gates [T, k] of float64 logits: the k largest, ties to the lower id."""
    ids = np.argsort(-l, axis=1, kind="stable")[:, :k]
    top = np.take_along_axis(l, ids, axis=1)
    z = np.exp(top - top[:, :1])
    return ids, z / z.sum(axis=1, keepdims=True)


def forward(x, ids, gates, get_expert, H, I, act="bf16"):
    """out [T, H], and a bound on the error of fp32 sums that keep h in two values of the type act.

    With u = 2^-23 the largest error of one (truncating) fp32 addition, a sum of n terms is off by at most n u times
    the sum of their sizes. Those of W13 go through silu (slope below 1.1) and the product into h; h is held to 2^-17
    (bf16) or 2^-21 (fp16) of itself, in fp16 also to 2^-38 of its token's largest; the sums of W2 add theirs; the
    gates are within 2e-6. No rounding of the result."""
    x = np.asarray(x, dtype=np.float64)
    T, k = ids.shape
    out, off = np.zeros((T, H)), np.zeros((T, H))
    u, split = 2.0 ** -23, 2.0 ** -17 if act == "bf16" else 2.0 ** -21
    for e in np.unique(ids):
        ex = get_expert(int(e))
        w13, w2 = (weights(ex["fmt"], *ex[n], K) for n, K in (("w13", H), ("w2", I)))
        for t, j in zip(*np.nonzero(ids == e)):
            gu, size = w13 @ x[t], np.abs(w13) @ np.abs(x[t])
            a, b = gu[:I], gu[I:]
            s = a / (1.0 + np.exp(-a))
            h = s * b
            da, db = (H + 16) * u * size[:I], (H + 16) * u * size[I:]
            dh = 1.1 * np.abs(b) * da + np.abs(s) * db + 1.1 * da * db + np.abs(h) * (split + 2.0 ** -20)
            if act == "f16":
                dh = dh + 2.0 ** -38 * np.abs(h).max()
            y, ysize = w2 @ h, np.abs(w2) @ np.abs(h)
            out[t] += gates[t, j] * y
            off[t] += gates[t, j] * (np.abs(w2) @ dh + ((2 * I + 16) * u + 2e-6 + 40 * u) * ysize)
    return out, off


def rms_tolerance(H, I, act="bf16"):
    """rms(error) / rms(result) of a token, of weights and x of random signs, where every sum, slot and digit of h is there.

    The result's rounding: half a step at most. A product of n terms: n / 16 MMAs and up to 32 joins and additions, each off
    by at most u = 2^-23 of a partial sum, whose rms is no larger than the whole sum's. W13's reaches h through silu'(a) b
    <= 1.1 |b| and silu(a), by up to 4 times itself (rms(a) / rms(silu(a)) <= 2). Then h's digits, expf and the gates."""
    u, half = 2.0 ** -23, 2.0 ** -8 if act == "bf16" else 2.0 ** -11
    split = 2.0 ** -17 if act == "bf16" else 2.0 ** -21
    return half + (4 * (H / 16 + 32) + I / 16 + 32) * u + split + 2.0 ** -18


def route_of(x, router, k, bias=None):
    return choose(logits(x, router, bias), k)


__all__ = ["weights", "logits", "choose", "forward", "rms_tolerance", "route_of", "route"]
