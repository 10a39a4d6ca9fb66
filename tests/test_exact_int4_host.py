"""What the exact integer linears reject, on the CPU."""

import numpy as np
import pytest

from oracle import int4 as oint4
from tests import exact_int4


@pytest.mark.parametrize("case", [c for c in exact_int4.CASES if c[1] * c[2] <= 1 << 26])
def test_a_lost_block_shows(case):
    L = exact_int4.ExactLinear(*case)
    want = L.result()
    ref = oint4.forward(L.x, L.codes, L.scales, L.zeros, L.group, L.bias)
    assert np.abs(ref - want).max() <= 2.0 ** -8 * np.abs(want).max()
    blocks = -(-case[2] // 128)
    for lost in {0, blocks // 3, blocks // 2, blocks - 2 if blocks > 1 else 0, blocks - 1}:
        assert (L.result(lost) != want).any()


def test_the_sum_bound_counts_no_weight_of_zero():
    L = exact_int4.ExactLinear(3, 20, 256, 64, True, "bf16")
    base = oint4.sum_bound(L.x, L.codes, L.scales, L.zeros, 64)
    k = 70
    keep = L.codes[:, k // 2] & 0xF0
    L.codes[:, k // 2] = keep | L.zeros[:, k // 64]
    L.x[:, k] = 0
    without = oint4.sum_bound(L.x, L.codes, L.scales, L.zeros, 64)
    L.x[:, k] = 1e9
    assert np.array_equal(oint4.sum_bound(L.x, L.codes, L.scales, L.zeros, 64), without) and (without <= base).all()
