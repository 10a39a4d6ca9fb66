"""GPU tests of the rows at the end of the 32-bit row index: 2^31 - 1 tokens of one value, one expert (34 GB)."""

import pytest
import torch

import nf3_moe_gb300 as hm

pytestmark = pytest.mark.gpu

T = 2 ** 31 - 1
STEP = 2 ** 28


def is_arange(t, n):
    flat = t.reshape(-1)
    return all(torch.equal(flat[a:min(a + STEP, n)], torch.arange(a, min(a + STEP, n), dtype=torch.int32, device="cuda"))
               for a in range(0, n, STEP))


@pytest.mark.parametrize("capacity", [0, 5000])
def test_the_last_row_index(capacity):
    desc = hm.DispatchDesc(1, 1, 1, hm.ROW_BF16, 1, capacity)
    R = hm.hmoe_dispatch_rows(desc, T)
    assert R == (capacity or T)
    x = torch.randn(STEP, device="cuda").to(torch.bfloat16).repeat(8)[:T].reshape(T, 1)
    perm = torch.arange(T, dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    rows = torch.full((R, 1), float("nan"), dtype=torch.bfloat16, device="cuda")
    row_slot = torch.full((R,), -77, dtype=torch.int32, device="cuda")
    slot_row = torch.full((T, 1), -77, dtype=torch.int32, device="cuda")
    row_offsets = torch.full((2,), -77, dtype=torch.int32, device="cuda")
    ws = torch.zeros(hm.hmoe_dispatch_workspace_size(desc, T), dtype=torch.uint8, device="cuda")
    try:
        hm.hmoe_dispatch(desc, x, perm, offsets, rows, row_slot, slot_row, row_offsets, ws)
        hm.hmoe_check_device_status(ws)
        assert row_offsets.tolist() == [0, R]
        assert is_arange(row_slot, R) and is_arange(slot_row, R)
        assert (slot_row[R:] == -1).all()
        assert torch.equal(rows, x[:R])
        out = torch.full((T, 1), float("nan"), dtype=torch.bfloat16, device="cuda")
        hm.hmoe_combine(desc, rows, slot_row, out, ws)
        hm.hmoe_check_device_status(ws)
        assert torch.equal(out[:R], x[:R]) and (out[R:] == 0).all()
    finally:
        del x, perm, rows, row_slot, slot_row
        torch.cuda.empty_cache()
