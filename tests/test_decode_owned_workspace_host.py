"""CPU tests of the workspace that HybridMoELayer makes for decode(): the layer is built over host memory, with the calls
that need a GPU replaced."""

import pytest
import torch

import nf3_moe_gb300 as hm


@pytest.fixture
def host_layer(monkeypatch):
    """HybridMoELayer(H, I, E, topk, ...) with host buffers; zeroed: the buffers that were zeroed, fail: an error for the n-th."""
    zeroed, fail = [], {}

    def init(ws, stream=None):
        zeroed.append(ws)
        if len(zeroed) in fail:
            raise fail[len(zeroed)]

    monkeypatch.setattr(hm, "hmoe_workspace_init", init)
    monkeypatch.setattr(hm, "hmoe_packed_size", lambda desc, bit_map: (16, 0))
    monkeypatch.setattr(hm, "hmoe_pack_weights", lambda *args: None)

    def make(H, I, E, topk, **kw):
        return hm.HybridMoELayer(H, I, E, topk, None, [], device="cpu", **kw)
    make.zeroed, make.fail = zeroed, fail
    return make


def test_as_many_tokens_as_the_sizes_admit(host_layer):
    """8 tokens of these sizes exceed the cost that a call can count, 7 do not: decode() is there for 7."""
    H, I = 39680, 19840
    layer = host_layer(H, I, 32, 32)
    assert layer.decode_ws.nbytes == hm.hmoe_decode_workspace_size(layer.desc, 7)
    assert host_layer.zeroed[-1] is layer.decode_ws
    with pytest.raises(hm.HmoeError) as ei:
        hm.hmoe_decode_workspace_size(layer.desc, 8)
    assert ei.value.status == -2


def test_no_more_than_asked_for(host_layer):
    for n in (1, 5, 8, 64):
        layer = host_layer(256, 128, 8, 2, max_tokens=n)
        assert layer.decode_ws.nbytes == hm.hmoe_decode_workspace_size(layer.desc, min(n, 8))


def test_a_layer_that_decode_does_not_take_says_why(host_layer):
    for layer in (host_layer(256, 128, 8, 2, act_globals=(1.0, 1.0)), host_layer(39680 + 128, 64, 8, 2)):
        assert layer.decode_ws is None
        with pytest.raises(hm.HmoeError) as ei:
            layer.decode(torch.zeros((1, layer.H), dtype=torch.bfloat16), torch.zeros((8, layer.H), dtype=torch.bfloat16))
        assert ei.value.status == -2


def test_an_error_of_the_zeroing_is_not_hidden(host_layer):
    host_layer.fail[2] = hm.HmoeError(-5, "launch")
    with pytest.raises(hm.HmoeError) as ei:
        host_layer(256, 128, 8, 2)
    assert ei.value.status == -5
