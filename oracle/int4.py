"""Oracle of the 4-bit integer linear: y = x W^T + bias, W = (q - z) s by groups along K. Float64 NumPy.

TEST INFRASTRUCTURE ONLY: see the package docstring.
"""

import numpy as np

from . import formats


def weights(codes, scales, zeros, group):
    """[N, K] from codes uint8 [N, K/2] (element 2i in the low nibble), scales and zeros [N, K/group] (None: 8)."""
    K = 2 * codes.shape[1]
    q = formats.unpack_nibbles(codes, K).astype(np.float64)
    z = np.full(scales.shape, 8.0) if zeros is None else (np.asarray(zeros) & 15).astype(np.float64)
    return (q - np.repeat(z, group, axis=1)) * np.repeat(np.asarray(scales, dtype=np.float64), group, axis=1)


def forward(x, codes, scales, zeros, group, bias=None):
    y = np.asarray(x, dtype=np.float64) @ weights(codes, scales, zeros, group).T
    return y if bias is None else y + np.asarray(bias, dtype=np.float64)


def bound(x, codes, scales, zeros, group, bias=None, act="bf16"):
    """A wide bound on the error of the sums alone. With u = 2^-23 the largest error of one fp32 addition: a group's sum of
    products, of terms up to 15 |x| in fp16 and 143 |x| in bf16 (room for products of 128 + q with the offset's share
    taken off the sum); then the sum over the groups of terms s |sum|, joined by up to 16 warps. sum_bound is what sums
    of the exact (q - z) x keep to."""
    x, s = np.abs(np.asarray(x, dtype=np.float64)), np.abs(np.asarray(scales, dtype=np.float64))
    T, K = x.shape
    u, groups = 2.0 ** -23, K // group
    per = x.reshape(T, groups, group).sum(axis=2)
    off = (143.0 * (2 * group + 16) if act == "bf16" else 15.0 * (group + 16)) * u * (per @ s.T)
    size = x @ np.abs(weights(codes, scales, zeros, group)).T
    return off + (2 * groups + 48) * u * (size + (0 if bias is None else np.abs(np.asarray(bias, dtype=np.float64))))


def sum_bound(x, codes, scales, zeros, group, bias=None):
    """A bound on the error of fp32 sums of the exact terms (q - z) x, whatever their offsets cost: with u = 2^-23 the
    largest error of one (truncating) fp32 addition, a group's sum of at most group + 16 additions, then as in bound().
    A weight of zero adds nothing, however large its x."""
    x = np.abs(np.asarray(x, dtype=np.float64))
    size = x @ np.abs(weights(codes, scales, zeros, group)).T
    groups = x.shape[1] // group
    return 2.0 ** -23 * ((group + 16 + 2 * groups + 48) * size + (2 * groups + 48) * (0 if bias is None else np.abs(np.asarray(bias, dtype=np.float64))))
