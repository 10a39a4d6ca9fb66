"""GPU tests of one batch in both of the kernels that a larger batch may go to, and of the tile kernels' sums over pieces.

The choice goes by the number of slots of the set, so the same adapters in a set of few and of many slots send the same
batch to the tile kernels and to the small one. Tolerance: as derived in test_gpu_lora.py (16 bits of A x in bf16, 22 in
fp16), for each side.
"""

import numpy as np
import pytest
import torch

import nf3_moe_gb300 as hm

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
BF, HF = torch.bfloat16, torch.float16
BITS = {BF: 8, HF: 11}
ACT = {BF: hm.ACT_BF16, HF: hm.ACT_F16}


def f64(t):
    return t.double().cpu().numpy()


def adapters_of(K, N, used, rank, dt, gen):
    made = []
    for i in range(used):
        r = rank if i == 0 else 1 + (7 * i * i + 3 * i) % rank
        A = (torch.randn((r, K), generator=gen, device="cuda") * K ** -0.5).to(dt)
        made.append((A, (torch.randn((N, r), generator=gen, device="cuda") * r ** -0.5).to(dt), 0.25 * (1 + i % 5)))
    return made


def launches(call):
    before = hm.hmoe_launch_count()
    out = call()
    return out, hm.hmoe_launch_count() - before


@pytest.mark.parametrize("shape", [(2300, 2056, 520, 5, 64, BF), (2300, 2056, 520, 5, 64, HF), (2300, 264, 136, 3, 32, BF), (2500, 1032, 72, 4, 16, HF)],
                         ids=str)
def test_the_same_batch_in_both_kernels(shape):
    T, K, N, used, rank, dt = shape
    gen = torch.Generator(device="cuda").manual_seed(T + K)
    made = adapters_of(K, N, used, rank, dt, gen)
    x, base = (torch.randn(s, generator=gen, device="cuda").to(dt) for s in ((T, K), (T, N)))
    ids = torch.randint(-1, used, (T,), generator=gen, device="cuda", dtype=torch.int32)
    ref, tol = f64(base), 6 * EPS * np.abs(f64(base)) + (2.0 ** -25 if dt == HF else 0.0)
    x64, at = f64(x), ids.cpu().numpy()
    for a, (A, B, s) in enumerate(made):
        rows, A, B = np.flatnonzero(at == a), f64(A), f64(B)
        u, absu = x64[rows] @ A.T, np.abs(x64[rows]) @ np.abs(A).T
        ref[rows] += s * (u @ B.T)
        du = (K / 16 + 16) * 2 * EPS * absu + 2.0 ** (-2 * BITS[dt]) * np.abs(u)
        tol[rows] += abs(s) * ((du + (A.shape[0] / 8 + 11) * 2 * EPS * np.abs(u)) @ np.abs(B).T)
    counts = []
    for slots in (used, 512):
        s = hm.LoraAdapters(K, N, slots, rank, max_tokens=T, act_dtype=ACT[dt])
        for a, (A, B, scale) in enumerate(made):
            s.load(a, A, B, scale)
        out, n = launches(lambda: s(x, ids, base=base))
        hm.hmoe_check_device_status(s.ws)
        assert (np.abs(f64(out) - ref) <= tol + 2.0 ** -BITS[dt] * np.abs(ref)).all()
        counts.append(n)
    assert counts == [3, 2]                               # plan, A x, B u; plan, small


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("shape", [(1600, 1032, 264, 3, 128), (2500, 2056, 520, 5, 96), (2300, 6152, 136, 4, 64)], ids=str)
def test_sums_over_pieces_give_the_same_bits(shape, dt):
    """K shared by several CTAs and rows scattered over the tiles: every pass sums in the same order."""
    T, K, N, slots, rank = shape
    gen = torch.Generator(device="cuda").manual_seed(T)
    s = hm.LoraAdapters(K, N, slots, rank, max_tokens=T, act_dtype=ACT[dt])
    for a, (A, B, scale) in enumerate(adapters_of(K, N, slots, rank, dt, gen)):
        s.load(a, A, B, scale)
    x, base = (torch.randn(sh, generator=gen, device="cuda").to(dt) for sh in ((T, K), (T, N)))
    ids = torch.randint(-1, slots, (T,), generator=gen, device="cuda", dtype=torch.int32)
    first, n = launches(lambda: s(x, ids, base=base))
    assert n == 3
    for _ in range(10):
        assert torch.equal(s(x, ids, base=base), first)
