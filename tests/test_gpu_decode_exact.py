"""The whole layer for a few tokens where no digit may be lost: exact layers, whose results have to equal the rounding of the
exact ones bit for bit, and the rms of the error of random layers (tests/test_exact_layer_host.py shows what both reject)."""

import numpy as np
import pytest
import torch

import synth
from oracle import decode as odec
from tests import exact_layer, gpu_util as U
from tests.test_gpu_decode import CASES as RANDOM_CASES, f64, make

pytestmark = pytest.mark.gpu

# the benchmark's two layers and a batch of one, beside the cases that the CPU checks too
LARGER = [(8, 6144, 2048, 32, 8, synth.FMT_NVFP4, 8, "bf16"), (1, 2048, 768, 128, 8, synth.FMT_NVFP4, None, "bf16"),
          (8, 128, 64, 512, 32, synth.FMT_NVFP4, 100, "bf16"),  # 256 slots of more experts than there are shares
          (8, 2048, 768, 64, 8, synth.FMT_NVFP4, None, "f16"), (4, 6144, 2048, 16, 8, synth.FMT_MXFP4, 4, "f16")]


@pytest.mark.parametrize("T,H,I,E,k,fmt,kept,act", exact_layer.CASES + LARGER)
def test_exact_layers_bit_for_bit(T, H, I, E, k, fmt, kept, act):
    L = exact_layer.ExactLayer(T, H, I, E, k, fmt, kept, act, device="cuda")
    moe = U.build(L.layer, T)
    x, router = (torch.from_numpy(v).cuda().to(moe.dtype) for v in (L.x, L.router))
    out, ids, gates = moe.decode(x, router)
    assert np.array_equal(ids.cpu().numpy(), L.ids)
    assert bool((gates == 1 / k).all())
    want = L.result()
    got = f64(out)
    assert np.array_equal(got, want), (np.argwhere(got != want)[:4], float(np.abs(got - want).max()))
    for t in {0, T // 2, T - 1}:                                   # alone, and beside others
        assert np.array_equal(f64(moe.decode(x[t:t + 1], router)[0])[0], want[t])


@pytest.mark.parametrize("T,H,I,E,k,fmt,kept,act", RANDOM_CASES)
def test_the_rms_of_random_layers(T, H, I, E, k, fmt, kept, act):
    L, moe, x, router = make(T, H, I, E, k, fmt, kept, act)
    out, ids, gates = moe.decode(x, router)
    want_ids, want_gates = odec.route_of(f64(x), f64(router), k)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    ref, _ = odec.forward(f64(x), want_ids, want_gates, L.expert_numpy, H, I, act)
    rms = lambda v: np.sqrt((v ** 2).mean(axis=1))  # noqa: E731
    # half a step of fp16's subnormals beside what is in proportion
    assert (rms(f64(out) - ref) <= odec.rms_tolerance(H, I, act) * rms(ref) + (2.0 ** -25 if act == "f16" else 0)).all()
