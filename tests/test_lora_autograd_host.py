"""CPU tests of what the adapters say to autograd (the library's call is replaced by a plain one): they have no gradient,
so a call that would lose one is refused, and what they write is seen as written."""

import pytest
import torch

import nf3_moe_gb300 as hm
from nf3_moe_gb300 import lora as lora_mod

K, N, T = 16, 24, 3


class _Lib:
    calls = 0

    def hmoe_lora_forward(self, *_):
        _Lib.calls += 1
        return 0


@pytest.fixture
def adapters(monkeypatch):
    a = hm.LoraAdapters.__new__(hm.LoraAdapters)
    a.desc, a.N, a.dtype, a.ws = hm.LoraDesc(K, N, 2, 4), N, torch.bfloat16, torch.zeros(512, dtype=torch.uint8)
    a.lora = type("Handle", (), {"handle": None, "desc": a.desc})()
    check = lora_mod._check_lora_forward
    monkeypatch.setattr(lora_mod, "_check_lora_forward", lambda *args: check(*args, cuda=False))
    monkeypatch.setattr(lora_mod._lib, "_LIB", _Lib())
    monkeypatch.setattr(lora_mod, "_raw_stream", lambda *_: 0)
    _Lib.calls = 0
    return a


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


ids = torch.zeros(T, dtype=torch.int32)


@pytest.mark.parametrize("what", ["x", "base", "out"])
def test_a_gradient_that_would_be_lost_is_refused(adapters, what):
    t = {"x": bf(T, K), "base": bf(T, N), "out": bf(T, N)}
    t[what] = t[what].requires_grad_() * 1                        # not a leaf
    with pytest.raises(RuntimeError, match=f"{what} requires a gradient"):
        adapters(t["x"], ids, base=t["base"], out=t["out"])
    assert _Lib.calls == 0                                        # nothing was launched
    with torch.no_grad():
        adapters(t["x"], ids, base=t["base"], out=t["out"])
    adapters(*(v.detach() for v in (t["x"], ids)), base=t["base"].detach(), out=t["out"].detach())
    assert _Lib.calls == 2


def test_what_they_write_counts_as_written(adapters):
    """A tensor that autograd keeps for a backward pass is changed in place: the backward pass says so."""
    w, y = torch.ones(T, N, dtype=torch.bfloat16, requires_grad=True), bf(T, N)
    loss = (w * y).sum()
    before = y._version
    adapters(bf(T, K), ids, base=y, out=y)
    assert y._version > before
    with pytest.raises(RuntimeError, match="inplace operation"):
        loss.backward()
    wide = bf(T, 2 * N)
    adapters(bf(T, K), ids, out=wide[:, :N])
    assert wide._version > 0
    with torch.inference_mode():                                  # such tensors keep no count
        y = bf(T, N)
        adapters(bf(T, K), ids, base=y, out=y)


def test_the_linear_refuses_before_it_writes(adapters):
    class Linear(hm.LinearW4A16):
        def __init__(self):
            self.linear, self.ws, self.N, self.dtype = None, None, N, torch.bfloat16

    x = bf(T, K).requires_grad_()
    with pytest.raises(RuntimeError, match="x requires a gradient"):
        Linear()(x, adapters=adapters, ids=ids)
