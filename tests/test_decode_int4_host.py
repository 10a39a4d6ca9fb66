"""CPU tests of the whole layer for a few tokens and of the 4-bit integer linear: sizes and refusals of the library,
and the binding's tensor checks."""

import ctypes

import pytest
import torch

import nf3_moe_gb300 as hm
from nf3_moe_gb300 import decode as dec_mod, int4 as int4_mod


@pytest.fixture(scope="module")
def lib():
    import os
    from nf3_moe_gb300 import _lib, build
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return _lib.lib()


def layer_desc(H=256, I=128, E=8, k=2, kept=hm.FMT_NVFP4, act=hm.ACT_BF16, quant=0):
    return hm.LayerDesc(H, I, E, k, kept, act, quant, 1.0, 1.0)


# ------------------------------------------------------------ the whole layer for a few tokens
def test_decode_workspace_sizes(lib):
    sizes = [hm.hmoe_decode_workspace_size(layer_desc(), t) for t in range(9)]
    assert sizes == sorted(sizes) and sizes[0] >= 256
    # a slot's h and result, fp32
    assert sizes[8] >= 8 * 2 * (128 + 256) * 4


@pytest.mark.parametrize("desc,T,status", [(layer_desc(), -1, -1), (layer_desc(), 9, -2), (layer_desc(quant=1), 1, -2),
                                           (layer_desc(H=100), 1, -2), (layer_desc(H=128 * 1024), 1, -2), (layer_desc(I=64 * 1024), 1, -2),
                                           (layer_desc(E=0), 1, -1), (layer_desc(k=9), 1, -2), (layer_desc(act=2), 1, -1)])
def test_decode_sizes_that_are_refused(lib, desc, T, status):
    with pytest.raises(hm.HmoeError) as ei:
        hm.hmoe_decode_workspace_size(desc, T)
    assert ei.value.status == status


def test_decode_null_arguments(lib):
    p = 4096                                         # never dereferenced
    assert lib.hmoe_decode(None, p, 1, p, None, p, None, None, p, 1 << 20, None) == -1
    assert lib.hmoe_decode_workspace_size(ctypes.byref(layer_desc()), 1, None) == -1


def test_decode_binding_checks():
    d, bf, i32, f32 = layer_desc(), torch.bfloat16, torch.int32, torch.float32
    ok = dict(x=torch.zeros(3, 256, dtype=bf), router=torch.zeros(8, 256, dtype=bf), out=torch.zeros(3, 256, dtype=bf),
              ids=torch.zeros(3, 2, dtype=i32), gates=torch.zeros(3, 2), ws=torch.zeros(512, dtype=torch.uint8), bias=torch.zeros(8))
    check = lambda **kw: dec_mod._check_decode(d, **(ok | kw), cuda=False)  # noqa: E731
    assert check()[0] == 3
    assert check(ids=None, gates=None, bias=None)[0] == 3
    for kw in (dict(x=torch.zeros(3, 255, dtype=bf)), dict(x=torch.zeros(3, 256)), dict(x=torch.zeros(256, dtype=bf)),
               dict(x=torch.zeros(256, 3, dtype=bf).t()), dict(x=torch.zeros(3, 512, dtype=bf)[:, :256]), dict(router=torch.zeros(7, 256, dtype=bf)),
               dict(router=torch.zeros(8, 256)), dict(out=torch.zeros(2, 256, dtype=bf)), dict(out=torch.zeros(3, 256)),
               dict(ids=torch.zeros(3, 2, dtype=torch.int64)), dict(ids=torch.zeros(3, 3, dtype=i32)), dict(gates=torch.zeros(3, 2, dtype=bf)),
               dict(gates=torch.zeros(2, 3).t()), dict(bias=torch.zeros(8, dtype=bf)), dict(bias=torch.zeros(9)),
               dict(ws=torch.zeros(512, dtype=torch.uint8)[::2])):
        with pytest.raises(ValueError):
            check(**kw)
    with pytest.raises(TypeError):
        check(x=[[0.0]])
    with pytest.raises(ValueError, match="CUDA"):    # host tensors never reach the library
        dec_mod._check_decode(d, **ok)


def test_decode_refuses_to_lose_a_gradient():
    for name in ("x", "router", "bias", "out", "gates"):
        with pytest.raises(RuntimeError, match=name):
            dec_mod._no_gradient(**{name: torch.zeros(2, requires_grad=True)})
    with torch.no_grad():
        dec_mod._no_gradient(x=torch.zeros(2, requires_grad=True))


# ------------------------------------------------------------ 4-bit integer linear
def test_int4_sizes(lib):
    # units of 16 rows, blocks of 128 along K: 1024 bytes of codes, 32 of scales a group, 16 of zero points
    assert hm.hmoe_int4_packed_size(hm.Int4Desc(17, 160, 32, 0, hm.ACT_BF16)) == 2 * 2 * (1024 + 4 * 32)
    assert hm.hmoe_int4_packed_size(hm.Int4Desc(16, 128, 128, 1, hm.ACT_F16)) == 1024 + 48
    assert hm.hmoe_int4_packed_size(hm.Int4Desc(1, 64, 64, 0, hm.ACT_BF16)) == 1024 + 2 * 32


@pytest.mark.parametrize("bad,status", [((0, 128, 128, 0, 0), -1), ((16, 0, 128, 0, 0), -1), ((16, 128, 128, 2, 0), -1), ((16, 128, 128, 0, 2), -1),
                                        ((16, 128, 16, 0, 0), -2), ((16, 128, 96, 0, 0), -2), ((16, 160, 64, 0, 0), -2),
                                        ((16, (1 << 20) + 128, 128, 0, 0), -2), (((1 << 20) + 1, 128, 128, 0, 0), -2), ((16, (1 << 31) - 128, 128, 0, 0), -2)])
def test_int4_bad_descriptors(lib, bad, status):
    with pytest.raises(hm.HmoeError) as ei:
        hm.hmoe_int4_packed_size(hm.Int4Desc(*bad))
    assert ei.value.status == status


def test_int4_null_arguments(lib):
    p = 4096                                         # never dereferenced
    assert lib.hmoe_int4_forward(None, p, 128, 1, None, p, 16, None) == -1
    d, h = hm.Int4Desc(16, 128, 128, 0, 0), ctypes.c_void_p()
    assert lib.hmoe_int4_pack(ctypes.byref(d), None, p, None, p, None, ctypes.byref(h)) == -1
    assert lib.hmoe_int4_pack(ctypes.byref(d), p, p, None, p + 16, None, ctypes.byref(h)) == -1
    assert b"128-byte" in lib.hmoe_last_error()
    assert lib.hmoe_int4_pack(ctypes.byref(d), p, p, p, p, None, ctypes.byref(h)) == -1   # zeros that the descriptor lacks
    z = hm.Int4Desc(16, 128, 128, 1, 0)
    assert lib.hmoe_int4_pack(ctypes.byref(z), p, p, None, p, None, ctypes.byref(h)) == -1
    assert lib.hmoe_int4_packed_size(ctypes.byref(d), None) == -1
    lib.hmoe_int4_destroy(None)


def test_int4_binding_checks(lib):
    d, bf, u8 = hm.Int4Desc(24, 128, 64, 1, hm.ACT_BF16), torch.bfloat16, torch.uint8
    ok = dict(x=torch.zeros(3, 128, dtype=bf), out=torch.zeros(3, 24, dtype=bf), bias=torch.zeros(24, dtype=bf))
    check = lambda **kw: int4_mod._check_int4_forward(d, **(ok | kw), cuda=False)  # noqa: E731
    assert check()[:3] == (3, 128, 24) and check(bias=None)[:3] == (3, 128, 24)
    wide = torch.zeros(3, 400, dtype=bf)
    assert check(x=wide[:, 8:136], out=wide[:, 300:324])[:3] == (3, 400, 400)
    assert check(x=wide[:1, :128], out=wide[:1, 300:324])[:3] == (1, 128, 24)
    for kw in (dict(x=torch.zeros(3, 127, dtype=bf)), dict(x=torch.zeros(3, 128)), dict(x=torch.zeros(128, 3, dtype=bf).t()),
               dict(x=torch.zeros(128, dtype=bf).expand(3, 128)), dict(out=torch.zeros(3, 25, dtype=bf)), dict(out=torch.zeros(2, 24, dtype=bf)),
               dict(out=torch.zeros(24, 3, dtype=bf).t()), dict(bias=torch.zeros(25, dtype=bf)), dict(bias=torch.zeros(24))):
        with pytest.raises(ValueError):
            check(**kw)
    with pytest.raises(TypeError):
        check(x=[[0.0]])
    with pytest.raises(ValueError, match="CUDA"):
        int4_mod._check_int4_forward(d, **ok)
    n = hm.hmoe_int4_packed_size(d)
    good = dict(codes=torch.zeros(24, 64, dtype=u8), scales=torch.zeros(24, 2, dtype=bf), zeros=torch.zeros(24, 2, dtype=u8),
                packed=torch.zeros(n, dtype=u8))
    int4_mod._check_int4_pack(d, **good, cuda=False)
    for kw in (dict(codes=torch.zeros(24, 63, dtype=u8)), dict(scales=torch.zeros(24, 2)), dict(scales=torch.zeros(24, 1, dtype=bf)),
               dict(zeros=torch.zeros(24, 2, dtype=torch.int32)), dict(packed=torch.zeros(n - 1, dtype=u8))):
        with pytest.raises(ValueError):
            int4_mod._check_int4_pack(d, **(good | kw), cuda=False)
    with pytest.raises(TypeError):
        int4_mod._check_int4_pack(d, **(good | dict(zeros=None)), cuda=False)
    with pytest.raises(ValueError):
        int4_mod._check_int4_pack(hm.Int4Desc(24, 128, 64, 0, hm.ACT_BF16), **good, cuda=False)


def test_int4_refuses_to_lose_a_gradient():
    a, b = torch.zeros(2), torch.zeros(2, requires_grad=True)
    for args in ((b, a, None), (a, b, None), (a, a, b)):
        with pytest.raises(RuntimeError, match="gradient"):
            int4_mod._no_gradient(*args)
    with torch.no_grad():
        int4_mod._no_gradient(b, a, None)
