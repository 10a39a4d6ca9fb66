"""GPU tests of the adapters at the ends of what their arguments may be."""

import ctypes

import pytest
import torch

import nf3_moe_gb300 as hm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [3.2e38, -3.4e38, 1e-44])
def test_every_finite_scale_is_taken(scale):
    a = hm.LoraAdapters(64, 64, 1, 1, max_tokens=4)
    A, B = torch.full((1, 64), 2.0 ** -6, device="cuda").bfloat16(), torch.full((64, 1), 2.0 ** -100, device="cuda").bfloat16()
    a.load(0, A, B, scale)
    x = torch.ones((4, 64), dtype=torch.bfloat16, device="cuda")
    out = a(x, torch.zeros(4, dtype=torch.int32, device="cuda"))
    want = (torch.tensor(scale, dtype=torch.float32).double() * 2.0 ** -100).to(torch.bfloat16).double()   # A x is 1
    assert ((out.double().cpu() - want).abs() <= 2.0 ** -7 * want.abs()).all()
    for bad in (float("inf"), -float("inf"), float("nan"), 3.5e38):
        with pytest.raises(hm.HmoeError) as ei:
            a.load(0, A, B, bad)
        assert ei.value.status == -1


def test_a_batch_above_the_limit_is_refused_before_anything_is_read():
    a = hm.LoraAdapters(8, 8, 1, 1, max_tokens=4)
    p = a.ws.data_ptr()
    status = hm._lib.lib().hmoe_lora_forward(a.lora.handle, p, 8, 2 ** 26 + 1, p, None, 0, p, 8, p, ctypes.c_size_t(256), None)
    assert status == -2
