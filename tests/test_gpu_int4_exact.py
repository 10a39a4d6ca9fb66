"""The 4-bit integer linear where no digit may be lost: exact inputs, whose results have to equal the rounding of the exact
ones bit for bit, and random ones under the bound that counts fp32 sums of the terms (q - z) x alone."""

import numpy as np
import pytest
import torch

import nf3_moe_gb300 as hm
from tests import exact_int4
from tests.test_gpu_int4 import ACT, DT, f64, make
from tests.test_gpu_int4_range import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,N,K,group,zeros,act", exact_int4.CASES)
def test_exact_inputs_bit_for_bit(T, N, K, group, zeros, act):
    L = exact_int4.ExactLinear(T, N, K, group, zeros, act)
    dev = lambda v, t: None if v is None else torch.from_numpy(v).cuda().to(t)  # noqa: E731
    linear = hm.LinearInt4(N, K, group, dev(L.codes, torch.uint8), dev(L.scales, DT[act]), dev(L.zeros, torch.uint8), act_dtype=ACT[act])
    x, bias = dev(L.x, DT[act]), dev(L.bias, DT[act])
    want, got = L.result(), f64(linear(x, bias=bias))
    assert np.array_equal(got, want), (np.argwhere(got != want)[:4], float(np.abs(got - want).max()))
    assert np.array_equal(f64(linear(x[T // 2:T // 2 + 1], bias=bias)), want[T // 2:T // 2 + 1])


@pytest.mark.parametrize("T,N,K", [(1, 2432, 6144), (1, 2432, 6272), (2, 2432, 6144), (3, 2432, 2048), (3, 2432, 2176), (8, 2448, 2048),
                                   (16, 2432, 2048), (16, 2432, 4096), (16, 4864, 8192), (16, 4880, 8192), (12, 2432, 6144)])
@pytest.mark.parametrize("act", ["bf16", "f16"])
def test_both_warp_counts_around_their_border(T, N, K, act):
    """152 units (or twice, and one more) of 16, 17, 48 or 49 blocks and up to 128: eight warps a CTA, or sixteen, with K whole or in parts."""
    test_exact_inputs_bit_for_bit(T, N, K, 128, True, act)


@pytest.mark.parametrize("T,K", [(1, 131072), (3, 32768), (16, 6144)])
def test_one_value_of_x_at_the_ends_of_each_block(T, K):
    """Rows of x with a single one: the weight there, wherever K is cut."""
    N, group = 40, 128
    L = exact_int4.ExactLinear(1, N, K, group, True, "bf16")
    linear = hm.LinearInt4(N, K, group, *(torch.from_numpy(v).cuda().to(t) for v, t in ((L.codes, torch.uint8), (L.scales, torch.bfloat16), (L.zeros, torch.uint8))))
    at = np.sort(np.concatenate([np.arange(0, K, 128), np.arange(127, K, 128)]))
    got = []
    for lo in range(0, len(at), T):
        ks = torch.from_numpy(at[lo:lo + T]).cuda()
        x = torch.zeros((len(ks), K), dtype=torch.bfloat16, device="cuda")
        x[torch.arange(len(ks), device="cuda"), ks] = 1
        got.append(linear(x))
    assert np.array_equal(f64(torch.cat(got)), L.w[:, at].T)


@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("T,N,K,group", [(1, 17, 256, 128), (5, 100, 640, 32), (8, 48, 512, 64), (16, 200, 2048, 128), (40, 40, 384, 64),
                                         (3, 16, 4544, 64), (16, 3000, 6144, 128), (1, 33, 131072, 128)])
def test_random_inputs_under_the_sums_own_bound(T, N, K, group, act):
    linear, x, (codes, scales, z, _) = make(T, N, K, group, act, True)
    check(linear(x), x, codes, scales, z, group, act)
