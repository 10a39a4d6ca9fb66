"""The decode step's example: every part against its oracle from the values that the part before it gave, eagerly and
from a replayed graph."""

import importlib.util
import os

import numpy as np
import pytest
import torch

import synth
from oracle import decode as odec, int4 as oint4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    at = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_step.py")
    spec = importlib.util.spec_from_file_location("example_decode_step", at)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def near(got, ref, off):
    assert (np.abs(f64(got) - ref) <= 2.0 ** -8 * (np.abs(ref) + off) + off).all()


def check(block, x, r):
    L = block.L
    for name, v, y in (("proj", x, r["y"]), ("head", r["h"], r["logits"])):
        codes, scales, zeros = block.packed[name]
        args = (f64(v), codes.cpu().numpy(), f64(scales), zeros.cpu().numpy(), 64)
        near(y, oint4.forward(*args), oint4.bound(*args))
    assert torch.equal(r["z"], x + r["y"]) and torch.equal(r["h"], r["z"] + r["m"])
    ids, gates = odec.route_of(f64(r["z"]), f64(block.router), L.topk, f64(block.bias))
    assert np.array_equal(r["ids"].cpu().numpy(), ids) and np.abs(f64(r["gates"]) - gates).max() <= 1e-6
    near(r["m"], *odec.forward(f64(r["z"]), ids, gates, L.expert_numpy, L.H, L.I))


def test_the_step(example):
    block = example.Block(4)
    x = synth.gen_x(4, block.L.H, device="cuda")
    check(block, x, block(x))
    graph, out = example.graph_of(block, x)
    for seed in (5, 6):
        x.copy_(synth.gen_x(4, block.L.H, seed=seed, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        check(block, x, out)
    for t in (1, 3):
        v = x[:t].clone()
        check(block, v, block(v))
