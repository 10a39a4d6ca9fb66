"""CPU pins of the oracles of the whole layer for a few tokens and of the 4-bit integer linear: scalar loops,
torch routines, and identities."""

import numpy as np
import torch

import synth
from oracle import decode as odec, formats, int4 as oint4, layer as olayer


def test_unrounded_weights():
    w = torch.randn((8, 128), generator=torch.Generator().manual_seed(1)) * 0.02
    for fmt in (synth.FMT_NVFP4, synth.FMT_MXFP4, synth.FMT_NF3):
        codes, scales, g = synth.quantise(fmt, w)
        c, s = codes.numpy(), scales.numpy().view(np.uint16) if fmt == synth.FMT_NF3 else scales.numpy()
        got = odec.weights(fmt, c, s, g, 128)
        if fmt == synth.FMT_NF3:
            cb = formats.nf3_codebook()
            for n in range(8):
                bits = int.from_bytes(c[n].tobytes(), "little")
                for k in range(128):
                    assert got[n, k] == cb[(bits >> (3 * k)) & 7] * float(scales.view(torch.bfloat16)[n, k // 64])
            assert np.array_equal(formats.bf16_rne(got), formats.dequant(fmt, c, s, g, 128))
        else:
            assert np.array_equal(got, formats.dequant(fmt, c, s, g, 128))


def test_choice_and_gates():
    g = np.random.default_rng(2)
    l = np.round(g.normal(size=(6, 20)), 1)                       # with ties
    ids, gates = odec.choose(l, 7)
    for t in range(6):
        want = sorted(range(20), key=lambda e: (-l[t, e], e))[:7]
        assert list(ids[t]) == want
        assert np.allclose(gates[t], torch.softmax(torch.tensor(l[t, want]), 0).numpy(), atol=1e-15)
    x, r, b = g.normal(size=(3, 5)), g.normal(size=(4, 5)), g.normal(size=4)
    assert np.allclose(odec.logits(x, r, b)[1, 2], sum(x[1, i] * r[2, i] for i in range(5)) + b[2])


def test_forward_is_the_layer_where_its_weights_are_exact():
    L = synth.make_layer(H=128, I=64, E=3, topk=2, kept=None)     # uniform NVFP4
    x = synth.gen_x(4, 128).float().numpy().astype(np.float64)
    ids, gates = np.array([[0, 1], [2, 0], [1, 2], [0, 2]]), np.full((4, 2), 0.5)
    out, off = odec.forward(x, ids, gates, L.expert_numpy, 128, 64)
    ref = olayer.moe_forward(x, ids, gates, L.expert_numpy, 128, 64)
    assert np.allclose(out, ref, rtol=1e-12, atol=1e-14)
    assert (off > 0).all() and off.max() < 1e-2 * np.abs(ref).max()  # a bound, and a useful one


def test_int4_by_hand():
    g = np.random.default_rng(3)
    q, z = g.integers(0, 16, (3, 64)), g.integers(0, 16, (3, 2))
    s, x, b = g.normal(size=(3, 2)), g.normal(size=(2, 64)), g.normal(size=3)
    codes = (q[:, 0::2] | q[:, 1::2] << 4).astype(np.uint8)
    for zeros in (None, z.astype(np.uint8), (z + 16).astype(np.uint8)):  # the low four bits count
        y = oint4.forward(x, codes, s, zeros, 32, b)
        for t in range(2):
            for n in range(3):
                want = sum(x[t, k] * (q[n, k] - (8 if zeros is None else z[n, k // 32])) * s[n, k // 32] for k in range(64)) + b[n]
                assert abs(y[t, n] - want) < 1e-12
    assert (oint4.bound(x, codes, s, None, 32, b) > 0).all()
    assert (oint4.bound(x, codes, s, None, 32, act="f16") < oint4.bound(x, codes, s, None, 32)).all()
