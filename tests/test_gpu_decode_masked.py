"""Router biases of minus infinity that leave a token fewer experts than its top-k, or none."""

import pytest
import torch

import nf3_moe_gb300 as hm
from tests.test_gpu_decode import check, make

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.mark.parametrize("T", [1, 5])
@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("left", [[7], [3, 38, 39], [0, 1, 2, 11, 12, 13, 20]])
def test_fewer_experts_than_top_k(left, act, T):
    """The experts that are left come first, then the lowest ids of the others, with gates of zero."""
    L, moe, x, router = make(T, 256, 64, 40, 8, kept=10, act=act)
    bias = torch.full((40,), -INF, device="cuda")
    bias[left] = 0.5
    got = moe.decode(x, router, bias=bias)
    check(L, moe, x, router, got, bias)
    rest = [e for e in range(40) if e not in left][:8 - len(left)]
    for t in range(T):
        assert sorted(got[1][t, :len(left)].tolist()) == left and got[1][t, len(left):].tolist() == rest
    assert not got[2][:, len(left):].any() and bool((got[2][:, :len(left)] > 0).all())


@pytest.mark.parametrize("act", ["bf16", "f16"])
def test_no_expert_left(act):
    """NaN gates and results over the lowest ids, as hmoe_plan_routes gives them, and the next call is as always."""
    L, moe, x, router = make(3, 256, 64, 40, 8, kept=10, act=act)
    out, ids, gates = moe.decode(x, router, bias=torch.full((40,), -INF, device="cuda"))
    want = torch.arange(8, device="cuda", dtype=torch.int32).expand(3, 8)
    assert torch.equal(ids, want) and bool(gates.isnan().all()) and bool(out.isnan().all())
    plan = moe.plan(torch.full((3, 40), -INF, device="cuda"))
    assert torch.equal(plan[0], want) and bool(plan[1].isnan().all())
    check(L, moe, x, router, moe.decode(x, router))


def test_one_token_without_an_expert_leaves_the_others():
    """Its logits overflow to minus infinity (x is finite); the others' do not."""
    L, moe, x, router = make(5, 256, 128, 6, 3, kept=3)            # few experts: the tokens share them
    router = router.abs() + 1
    x[2] = -3e38
    out, ids, gates = moe.decode(x, router)
    assert bool(gates[2].isnan().all()) and bool(out[2].isnan().all()) and ids[2].tolist() == [0, 1, 2]
    clean = x.clone()
    clean[2] = 0
    keep = [0, 1, 3, 4]
    check(L, moe, clean, router, (out, ids, gates), rows=keep)
    hm.hmoe_check_device_status(moe.decode_ws)
