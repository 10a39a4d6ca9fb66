"""CPU tests of the low-rank adapters: sizes and refusals of the library and the binding's tensor checks."""

import ctypes

import pytest
import torch

import nf3_moe_gb300 as hm
from nf3_moe_gb300 import lora as lora_mod


@pytest.fixture(scope="module")
def lib():
    import os
    from nf3_moe_gb300 import _lib, build
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return _lib.lib()


def test_sizes(lib):
    # rank 13 is held as 16; K = 72 takes two 64-wide tiles, N = 64 one: 3 tiles of 16 x 128 bytes a slot, and the tables
    assert hm.hmoe_lora_packed_size(hm.LoraDesc(72, 64, 5, 13)) == 2 * 256 + 5 * 3 * 16 * 128
    assert hm.hmoe_lora_packed_size(hm.LoraDesc(64, 64, 65, 16)) == 2 * 512 + 65 * 2 * 16 * 128
    d = hm.LoraDesc(2048, 2048, 16, 16)
    sizes = [hm.hmoe_lora_workspace_size(d, t) for t in (0, 1, 8, 64, 4096)]
    assert sizes == sorted(sizes) and sizes[0] >= 256


@pytest.mark.parametrize("bad,status", [((0, 64, 1, 1), -1), ((64, 0, 1, 1), -1), ((64, 64, 0, 1), -1), ((64, 64, 1, 0), -1),
                                        ((64, 64, 1, 1, 2), -1), ((60, 64, 1, 1), -2), ((64, 60, 1, 1), -2), ((64, 64, 513, 1), -2),
                                        ((64, 64, 1, 129), -2), ((131080, 64, 1, 1), -2)])
def test_bad_descriptors_are_refused(lib, bad, status):
    for call in (lambda: hm.hmoe_lora_packed_size(hm.LoraDesc(*bad)), lambda: hm.hmoe_lora_workspace_size(hm.LoraDesc(*bad), 8)):
        with pytest.raises(hm.HmoeError) as ei:
            call()
        assert ei.value.status == status


def test_null_handles_are_refused(lib):
    p = 4096                                         # never dereferenced
    assert lib.hmoe_lora_forward(None, p, 64, 1, p, None, 0, p, 64, p, 256, None) == -1
    assert lib.hmoe_lora_load(None, 0, p, p, 1, ctypes.c_float(1.0), None) == -1
    d, h = hm.LoraDesc(64, 64, 1, 1), ctypes.c_void_p()
    assert lib.hmoe_lora_create(ctypes.byref(d), None, None, ctypes.byref(h)) == -1
    assert lib.hmoe_lora_create(ctypes.byref(d), 4104, None, ctypes.byref(h)) == -1
    assert b"256-byte" in lib.hmoe_last_error()
    with pytest.raises(hm.HmoeError):
        hm.hmoe_lora_workspace_size(d, -1)
    lib.hmoe_lora_destroy(None)


def test_binding_checks(lib):
    d = hm.LoraDesc(64, 128, 4, 8)
    bf = torch.bfloat16
    ok = dict(x=torch.zeros(3, 64, dtype=bf), ids=torch.zeros(3, dtype=torch.int32), base=torch.zeros(3, 128, dtype=bf),
              out=torch.zeros(3, 128, dtype=bf), ws=torch.zeros(512, dtype=torch.uint8))
    check = lambda **kw: lora_mod._check_lora_forward(d, **(ok | kw), cuda=False)  # noqa: E731
    assert check()[:4] == (3, 64, 128, 128)
    assert check(base=None)[:4] == (3, 64, 0, 128)
    wide = torch.zeros(3, 400, dtype=bf)
    assert check(base=wide[:, 16:144], out=wide[:, 160:288])[:4] == (3, 64, 400, 400)
    one = {"x": torch.zeros(1, 64, dtype=bf), "ids": torch.zeros(1, dtype=torch.int32), "base": None, "out": torch.zeros(400, dtype=bf)[8:136][None]}
    assert check(**one)[0] == 1
    for kw in (dict(x=torch.zeros(3, 63, dtype=bf)), dict(x=torch.zeros(3, 64)), dict(x=torch.zeros(64, 3, dtype=bf).t()),
               dict(x=torch.zeros(64, dtype=bf).expand(3, 64)), dict(ids=torch.zeros(3, dtype=torch.int64)),
               dict(ids=torch.zeros(4, dtype=torch.int32)), dict(base=torch.zeros(2, 128, dtype=bf)), dict(out=torch.zeros(3, 136, dtype=bf)),
               dict(out=torch.zeros(3, 128, dtype=torch.float16))):
        with pytest.raises(ValueError):
            check(**kw)
    with pytest.raises(TypeError):
        check(x=[[0.0]])
    with pytest.raises(ValueError):
        lora_mod._check_lora_load(d, 0, torch.zeros(8, 64, dtype=bf), torch.zeros(128, 7, dtype=bf), cuda=False)
    with pytest.raises(ValueError):
        lora_mod._check_lora_load(d, 0, torch.zeros(8, 63, dtype=bf), torch.zeros(128, 8, dtype=bf), cuda=False)
