"""CPU tests: calls without a derivative refuse tensors that carry a forward-mode one, which does not show in requires_grad
and which torch.no_grad() does not stop."""

from types import SimpleNamespace

import pytest
import torch
from torch.autograd import forward_ad

import nf3_moe_gb300 as hm
from nf3_moe_gb300 import decode as dec_mod, int4 as int4_mod, lora as lora_mod, rows as rows_mod


def test_the_level_that_is_looked_at():
    assert not rows_mod._forward_mode()
    with forward_ad.dual_level():
        assert rows_mod._forward_mode()
    assert not rows_mod._forward_mode()


NONE = SimpleNamespace(handle=None, desc=None)   # the library refuses it, should it be reached


def _decode(t):
    dec_mod.hmoe_decode(NONE, t["x"], t["router"], t["out"], t["ws"], t["bias"], t["ids"], t["gates"], stream=SimpleNamespace(cuda_stream=None))


def _int4(t):
    int4_mod.hmoe_int4_forward(NONE, t["x"], t["out"], t["bias"], stream=SimpleNamespace(cuda_stream=None))


def _lora(t):
    lora_mod.hmoe_lora_forward(NONE, t["x"], t["ids"], t["out"], t["ws"], base=t["base"], stream=SimpleNamespace(cuda_stream=None))


@pytest.mark.parametrize("call,names", [(_decode, ("x", "router", "out", "bias", "gates")), (_int4, ("x", "out", "bias")), (_lora, ("x", "out", "base"))])
def test_dual_tensors_are_refused(monkeypatch, call, names):
    monkeypatch.setattr(dec_mod, "_check_decode", lambda *args: (1, 0))
    monkeypatch.setattr(int4_mod, "_check_int4_forward", lambda *args: (1, 8, 8, 0))
    monkeypatch.setattr(lora_mod, "_check_lora_forward", lambda *args: (1, 8, 8, 8, 0))
    made = {n: torch.zeros(8) for n in ("x", "router", "out", "bias", "gates", "base", "ids", "ws")}
    for name in names:
        for quiet in (torch.no_grad, torch.enable_grad):
            with forward_ad.dual_level(), quiet():
                dual = forward_ad.make_dual(made[name], torch.ones(8))
                with pytest.raises(RuntimeError, match=f"{name} carries a forward-mode derivative"):
                    call(made | {name: dual})
                with pytest.raises(hm.HmoeError, match="is NULL"):   # its primal goes on to the library
                    call(made | {name: forward_ad.unpack_dual(dual).primal})

