"""The 4-bit integer linear where x spans a wide range: values far above the others, infinities, bf16's upper end.

Tolerance: oracle.int4.sum_bound, which counts the rounding of fp32 sums of the exact terms (q - z) x and nothing for
weights of zero, plus half a step of the result's type (2^-8 of the value in bf16, 2^-11 in fp16).
"""

import numpy as np
import pytest
import torch

import nf3_moe_gb300 as hm
from oracle import int4 as oint4

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
ACT = {"bf16": hm.ACT_BF16, "f16": hm.ACT_F16}
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def make(T, N, K, group, act, zeros, scale=0.005, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 13 * T + N)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = (scale * (0.5 + torch.rand((N, K // group), generator=g, device="cuda"))).to(DT[act])
    z = torch.randint(0, 16, (N, K // group), generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    return codes, scales, z, torch.randn((T, K), generator=g, device="cuda").to(DT[act])


def set_code(codes, k, q):
    """Every row's code at k."""
    keep = codes[:, k // 2] & (0xF0 if k % 2 == 0 else 0x0F)
    codes[:, k // 2] = keep | (q << (4 * (k % 2))).to(torch.uint8)


def check(out, x, codes, scales, z, group, act):
    args = (f64(x), codes.cpu().numpy(), f64(scales), None if z is None else z.cpu().numpy(), group)
    ref, off = oint4.forward(*args), oint4.sum_bound(*args)
    err = np.abs(f64(out) - ref)
    assert (err <= HALF[act] * (np.abs(ref) + off) + off + (2.0 ** -25 if act == "f16" else 0.0)).all(), float(err.max())


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("T,N,K,group", [(4, 512, 2048, 128), (3, 100, 1056, 32), (12, 64, 6144, 64)])
@pytest.mark.parametrize("act,far", [("bf16", 1e3), ("bf16", 1e5), ("bf16", 1e7), ("bf16", 1e30), ("f16", 1e3), ("f16", 6e4)])
def test_a_far_value_on_a_weight_of_zero(act, far, T, N, K, group, zeros):
    """The result is that of the other values alone, to the rounding of their own sums."""
    codes, scales, z, x = make(T, N, K, group, act, zeros)
    for k in (3, K // 2, K - 2):
        set_code(codes, k, torch.full((N,), 8, device="cuda") if z is None else z[:, k // group])
        x[:, k] = far
    out = hm.LinearInt4(N, K, group, codes, scales, z, act_dtype=ACT[act])(x)
    check(out, x, codes, scales, z, group, act)


@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("zeros", [False, True])
def test_infinities_follow_the_weights(act, zeros):
    """An infinite x gives the weight's sign times it, and NaN where the weight is zero or two infinities meet."""
    N, K, group = 96, 512, 64
    codes, scales, z, x = make(6, N, K, group, act, zeros)
    x[1, 100], x[2, 7] = float("inf"), float("-inf")
    x[4, 9], x[4, 300] = float("inf"), float("-inf")
    out = f64(hm.LinearInt4(N, K, group, codes, scales, z, act_dtype=ACT[act])(x))
    with np.errstate(invalid="ignore"):
        w = oint4.weights(codes.cpu().numpy(), f64(scales), None if z is None else z.cpu().numpy(), group)
        for t, at in ((1, [100]), (2, [7]), (4, [9, 300])):
            want = sum(f64(x)[t, k] * w[:, k] for k in at)
            assert np.array_equal(out[t], want, equal_nan=True)
            assert np.isinf(want).any() and np.isnan(want).any()
    keep = [0, 3, 5]
    check(torch.from_numpy(out[keep]), x[keep], codes, scales, z, group, act)


def test_the_upper_end_of_bf16():
    """x to 2^116: a group's sum before its scale is at most 128 x 15 x 2^116 < 2^127."""
    N, K, group = 64, 1024, 128
    codes, scales, z, x = make(4, N, K, group, "bf16", True, scale=2.0 ** -30)
    x = (x.float().clamp(-1, 1) * 2.0 ** 116).bfloat16()
    check(hm.LinearInt4(N, K, group, codes, scales, z)(x), x, codes, scales, z, group, "bf16")
