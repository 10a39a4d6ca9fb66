"""CPU tests of the adapters' limits: batches that the plan's row words do not hold are refused."""

import pytest

import nf3_moe_gb300 as hm

MOST = 2 ** 26  # a plan word has 10 bits for the group and 21 for the place in a warp's 32nd part of the rows


@pytest.fixture(scope="module", autouse=True)
def lib():
    import os
    from nf3_moe_gb300 import _lib, build
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return _lib.lib()


def test_the_plan_word_holds_every_place_up_to_the_limit():
    """The largest place of a warp's range beside the largest group stays a positive 32-bit number at the limit, and
    does not above it."""
    def largest(T):
        rounds = -(-T // 1024)
        return (rounds * 32 - 1) << 10 | 512
    assert largest(MOST) < 2 ** 31 <= largest(MOST + 1)


@pytest.mark.parametrize("T", [MOST + 1, 70_000_000, 2 ** 31 - 1])
def test_larger_batches_are_refused(T):
    d = hm.LoraDesc(8, 8, 4, 8)
    assert hm.hmoe_lora_workspace_size(d, MOST) > 0
    with pytest.raises(hm.HmoeError) as ei:
        hm.hmoe_lora_workspace_size(d, T)
    assert ei.value.status == -2


@pytest.mark.parametrize("rank", [16, 64, 128])
def test_batches_of_one_launch_need_no_scratch(rank):
    """Up to 128 rows a batch keeps nothing outside its one kernel: a server's workspace for a decode step is small."""
    d = hm.LoraDesc(2048, 2048, 16, rank)
    sizes = [hm.hmoe_lora_workspace_size(d, T) for T in (0, 1, 8, 128, 129, 4096)]
    assert sizes == sorted(sizes)
    assert sizes[0] >= 256 and sizes[3] <= 4096
    assert sizes[4] >= 2 * 129 * 4
