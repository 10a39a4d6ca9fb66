"""What the two GPU criteria of the whole layer for a few tokens reject: the exact layers' equality and the rms of random
ones. Each mistake is planted in the float64 oracle, on the CPU."""

import numpy as np
import pytest

import synth
from oracle import decode as odec, formats
from tests import exact_layer
from tests.test_gpu_decode import CASES as RANDOM_CASES


def _one_value(act):
    """h as one value of the type (fp16: its 11 digits, in a range of its own)."""
    return (lambda h: formats.bf16_rne(h)) if act == "bf16" else (lambda h: formats.f16_rne(h / 16) * 16)


@pytest.mark.parametrize("case", exact_layer.CASES)
def test_equality_rejects(case):
    L = exact_layer.ExactLayer(*case)
    ids, gates = odec.route_of(L.x, L.router, L.k)
    assert np.array_equal(ids, L.ids) and (gates == 1 / L.k).all()
    want = L.result()
    if L.H * L.I <= 1 << 19:                                       # the same by the formats' own oracle
        ref, _ = odec.forward(L.x, ids, gates, L.layer.expert_numpy, L.H, L.I, L.act)
        assert np.abs(ref - want).max() <= 2.0 ** -8 * np.abs(want).max()
    last13, last2 = L.H // 64 - 1, L.I // 64 - 1
    wrong = [L.result(drop_slot=True), L.result(drop13=0), L.result(drop13=last13 // 2), L.result(drop13=last13),
             L.result(drop2=0), L.result(drop2=last2 // 2), L.result(drop2=last2)]
    for w in wrong:
        assert (w != want).any(axis=1).all()                       # in every token
    # fp16 holds the h of small layers in one value
    h = max(np.abs(L.x @ w.T[:, :L.I].astype(np.float64) * (L.x @ w.T[:, L.I:].astype(np.float64))).max() for w in L.w13.values())
    if L.act == "bf16" or h >= 2 ** 12:
        assert (L.result(h_of=_one_value(L.act)) != want).any()


def _random(T, H, I, E, k, fmt, kept, act):
    L = synth.make_layer(H=H, I=I, E=E, topk=k, kept_ids=None if kept is None else list(range(0, E, max(1, E // max(1, kept))))[:kept],
                         uniform=kept is None, kept_format=fmt, act=act)
    r = np.random.default_rng(T + H + I)
    x = formats.act_rne(r.normal(size=(T, H)).astype(np.float32).astype(np.float64), act)
    router = formats.act_rne((r.normal(size=(E, H)) * H ** -0.5).astype(np.float32).astype(np.float64), act)
    return L, x, router


@pytest.mark.parametrize("T,H,I,E,k,fmt,kept,act", [c for c in RANDOM_CASES if c[3] < 512 and c[1] * c[2] * c[3] <= 1 << 24])
def test_the_rms_rejects(T, H, I, E, k, fmt, kept, act):
    L, x, router = _random(T, H, I, E, k, fmt, kept, act)
    ids, gates = odec.route_of(x, router, k)
    held = {}

    def run(drop_slot=False, drop13=None, drop2=None):
        out = np.zeros((T, H))
        for t in range(T):
            for j in range(1 if drop_slot else 0, k):
                e = int(ids[t, j])
                if e not in held:
                    ex = L.expert_numpy(e)
                    held[e] = [odec.weights(ex["fmt"], *ex[n], K) for n, K in (("w13", H), ("w2", I))]
                w13, w2 = held[e]
                v = x[t].copy()
                if drop13 is not None:
                    v[64 * drop13:64 * drop13 + 64] = 0
                gu = w13 @ v
                h = gu[:I] / (1 + np.exp(-gu[:I])) * gu[I:]
                if drop2 is not None:
                    h[64 * drop2:64 * drop2 + 64] = 0
                out[t] += gates[t, j] * (w2 @ h)
        return out
    ref = run()
    tol = odec.rms_tolerance(H, I, act)
    rms = lambda v: np.sqrt((v ** 2).mean(axis=1))  # noqa: E731
    assert (rms(formats.act_rne(ref.astype(np.float32).astype(np.float64), act) - ref) <= tol * rms(ref)).all()
    for wrong in (run(drop_slot=True), run(drop13=H // 64 - 1), run(drop2=I // 64 - 1), 0 * ref):
        assert (rms(wrong - ref) > 2 * tol * rms(ref)).all()
