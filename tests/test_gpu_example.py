"""The example's two paths against the oracles: a projection with adapters of many requests, and the MoE layer
with a low-rank branch for every expert and its gradients."""

import numpy as np
import pytest
import torch

import nf3_moe_gb300 as hm
from oracle import lora as olora
from oracle import rows as orows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    import importlib.util
    import os
    at = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "adapters.py")
    spec = importlib.util.spec_from_file_location("example_adapters", at)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def f64(t):
    return t.detach().double().cpu().numpy()


def test_projection_with_adapters(example):
    x, ids, weights, plain, y = example.serve()
    adapters = {a: (f64(A), f64(B), s) for a, (A, B, s) in weights.items()}
    ref = olora.forward(f64(x), ids.cpu().numpy(), adapters, f64(plain))
    # one rounding to bf16 of the exact sum, and fp32 sums of 512 and 16 terms
    size = olora.forward(np.abs(f64(x)), ids.cpu().numpy(), {a: (np.abs(A), np.abs(B), s) for a, (A, B, s) in adapters.items()},
                         np.abs(f64(plain)))
    assert (np.abs(f64(y) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -15 * size).all()
    none = (ids == -1).cpu().numpy()
    assert none.any() and np.array_equal(f64(y)[none], f64(plain)[none])


def test_expert_branch_and_its_gradients(example):
    r = example.expert_branch()
    ids, gates, perm, offsets = r["routes"]
    E, k = len(r["weights"]), ids.shape[1]
    row_slot, slot_row, _ = orows.row_maps(ids.cpu().numpy(), E)
    assert np.array_equal(r["plan"].slot_row.cpu().numpy(), slot_row)
    rows = orows.dispatch(f64(r["x"]), row_slot, k)
    expert = ids.cpu().numpy().reshape(-1)[row_slot]
    adapters = {e: (f64(A), f64(B), 1.0) for e, (A, B) in enumerate(r["weights"])}
    z = olora.forward(rows, expert, adapters, N=rows.shape[1])
    assert np.abs(f64(r["z"]) - z).max() <= 2.0 ** -7 * np.abs(z).max()
    # from the rows that the branch had: the gate-weighted sum, joined by torch in bf16
    g = f64(gates)
    delta = orows.combine(f64(r["z"]), slot_row, g)
    ref = f64(r["frozen"]) + delta
    assert (np.abs(f64(r["y"]) - ref) <= 2.0 ** -8 * (np.abs(ref) + np.abs(delta)) + 2.0 ** -16).all()
    dz = orows.dispatch(f64(r["dy"]), row_slot, k, g)
    assert (np.abs(f64(r["z"].grad) - dz) <= (2.0 ** -8 + 2.0 ** -24) * np.abs(dz)).all()
    dg, size = orows.gate_grads(f64(r["z"]), f64(r["dy"]), slot_row)
    dl = orows.logit_grads(dg, g, ids.cpu().numpy(), E)
    assert np.abs(f64(r["logits"].grad) - dl).max() <= 2.0 ** -18 * size.max()


def test_linear_takes_adapters_of_other_widths_only_with_an_error(example):
    x, ids, _, _, _ = example.serve()
    import synth
    codes, scales, g = synth.quant_nvfp4(0.02 * torch.randn((256, 512), device="cuda"))
    linear = hm.LinearW4A16(256, 512, hm.FMT_NVFP4, codes, scales, g, max_tokens=24)
    with pytest.raises(ValueError):
        linear(x, adapters=hm.LoraAdapters(512, 384, 2, 4, max_tokens=24), ids=ids)
