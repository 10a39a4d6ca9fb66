"""CPU tests: sizes and strides that a 32-bit argument of the library does not hold are refused by the binding (ctypes
would pass their low 32 bits, and a few rows, or rows elsewhere, would be taken for the whole). The tensors are on the
meta device: no memory."""

import pytest
import torch

import nf3_moe_gb300 as hm
from nf3_moe_gb300 import lora as lora_mod
from nf3_moe_gb300 import rows as rows_mod

BF, I32 = torch.bfloat16, torch.int32
WRAPS = 2 ** 32 + 4                                  # the low 32 bits are 4


def meta(*shape, dtype=BF):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.fixture(scope="module", autouse=True)
def lib():
    import os
    from nf3_moe_gb300 import _lib, build
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return _lib.lib()


@pytest.mark.parametrize("what", ["x", "base", "out"])
def test_row_strides_of_the_adapters(what):
    d = hm.LoraDesc(64, 64, 4, 8)
    t = {"x": meta(3, 64), "base": meta(3, 64), "out": meta(3, 64)}
    ids, ws = meta(3, dtype=I32), meta(512, dtype=torch.uint8)
    for ld, fits in ((2 ** 31 - 8, True), (2 ** 31, False), (2 ** 32 + 64, False)):
        t[what] = torch.empty_strided((3, 64), (ld, 1), dtype=BF, device="meta")
        if fits:
            assert ld in lora_mod._check_lora_forward(d, t["x"], ids, t["base"], t["out"], ws, cuda=False)[1:4]
            continue
        with pytest.raises(ValueError, match=what):
            lora_mod._check_lora_forward(d, t["x"], ids, t["base"], t["out"], ws, cuda=False)
    t[what] = torch.empty_strided((1, 64), (2 ** 32 + 64, 1), dtype=BF, device="meta")     # one row: its stride is never used
    t = {k: v if k == what else meta(1, 64) for k, v in t.items()}
    assert lora_mod._check_lora_forward(d, t["x"], meta(1, dtype=I32), t["base"], t["out"], ws, cuda=False)[1:4] == (64, 64, 64)


def test_rows_of_the_adapters():
    d = hm.LoraDesc(8, 8, 4, 8)
    with pytest.raises(ValueError, match="x"):
        lora_mod._check_lora_forward(d, meta(WRAPS, 8), meta(WRAPS, dtype=I32), None, meta(WRAPS, 8), meta(512, dtype=torch.uint8), cuda=False)


def test_tokens_of_the_rows():
    d = hm.DispatchDesc(8, 4, 1, hm.ROW_BF16, 1, 0)
    T, ws = WRAPS, meta(256, dtype=torch.uint8)
    with pytest.raises(ValueError, match="x"):
        rows_mod._check_dispatch(d, meta(T, 8), meta(T, dtype=I32), meta(5, dtype=I32), meta(T, 8), meta(T, dtype=I32),
                                 meta(T, 1, dtype=I32), meta(5, dtype=I32), ws, None, cuda=False)
    with pytest.raises(ValueError, match="out"):
        rows_mod._check_collect(d, "rows", meta(T, 8), meta(T, 1, dtype=I32), "out", meta(T, 8), ws, None, cuda=False)


@pytest.mark.parametrize("call", [lambda n: hm.hmoe_dispatch_rows(hm.DispatchDesc(8, 4, 1, 0, 1, 0), n),
                                  lambda n: hm.hmoe_dispatch_workspace_size(hm.DispatchDesc(8, 4, 1, 0, 1, 0), n),
                                  lambda n: hm.hmoe_lora_workspace_size(hm.LoraDesc(8, 8, 4, 8), n)])
def test_sizes_asked_for(call):
    call(4)
    for n in (WRAPS, -2 ** 32 + 4, 2 ** 31):
        with pytest.raises((ValueError, hm.HmoeError)):
            call(n)
