"""GPU tests of fp16 adapters whose A x leaves the middle of fp16's range: far below 1, above 65504, of very different
sizes in one batch and in one row, and infinite.

Tolerance of an output (e = 2^-24, r the rank, u = A x): u is summed in fp32 in chains of at most K / 16 + 16 steps, each
at most 2 e of the sum of absolute terms. It enters the second product with 22 bits, 2^-22 |u|, and with a floor for the
whole row, whose largest |u| is brought to 2^14 at least and then held to 2^-25: 2^-39 of a bound on that largest |u|.
The bound is the largest piece's times the pieces, at most K / 256 + 2 of them. The second product adds r / 8 + 8 steps,
the scale and the base 3 more; the result is rounded once, 2^-11, and 2^-25 for subnormals.
"""

import numpy as np
import pytest
import torch

import nf3_moe_gb300 as hm

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
HF = torch.float16

SHAPES = [  # T, K, N, slots, max_rank: batches of each of the ways that a batch may go
    (1, 512, 264, 1, 16), (5, 1000, 256, 3, 33), (100, 264, 520, 4, 64), (300, 1000, 264, 5, 64), (300, 328, 136, 3, 128),
    (3000, 136, 520, 512, 16), (2300, 2056, 520, 5, 64), (1600, 1032, 264, 3, 128), (2500, 72, 72, 2, 48)]


def f64(t):
    return t.double().cpu().numpy()


class Batch:
    def __init__(self, shape, a_std=1.0, b_std=1.0, scale=1.0, by_rank=False):
        T, K, N, slots, most = shape
        self.T, self.K, self.N, self.slots = T, K, N, slots
        self.gen = g = torch.Generator(device="cuda").manual_seed(T + K)
        self.hm = hm.LoraAdapters(K, N, slots, most, max_tokens=T, act_dtype=hm.ACT_F16)
        self.of = []
        for i in range(slots):
            r = most if i == 0 else 1 + (7 * i * i + 3 * i) % most
            by = 2.0 ** (torch.arange(r, device="cuda") % 12) if by_rank else torch.ones(r, device="cuda")
            A = (torch.randn((r, K), generator=g, device="cuda") * (a_std * K ** -0.5) / by[:, None]).to(HF)
            B = (torch.randn((N, r), generator=g, device="cuda") * (b_std * r ** -0.5) * by[None, :] / by.max()).to(HF)
            self.hm.load(i, A, B, scale)
            self.of.append((f64(A), f64(B), scale))
        self.ids = torch.randint(0, slots, (T,), generator=g, device="cuda", dtype=torch.int32)

    def randn(self, *shape):
        return torch.randn(shape, generator=self.gen, device="cuda")

    def run_and_check(self, x, base=None):
        out = torch.full((self.T, self.N), float("nan"), dtype=HF, device="cuda")
        self.hm(x, self.ids, base=base, out=out)
        hm.hmoe_check_device_status(self.hm.ws)
        ids, x64 = self.ids.cpu().numpy(), f64(x)
        ref = np.zeros((self.T, self.N)) if base is None else f64(base)
        tol = 6 * EPS * np.abs(ref) + 2.0 ** -25
        for a in np.unique(ids):
            A, B, s = self.of[a]
            at, r = np.flatnonzero(ids == a), A.shape[0]
            u, absu = x64[at] @ A.T, np.abs(x64[at]) @ np.abs(A).T
            du = (self.K / 16 + 16) * 2 * EPS * absu + 2.0 ** -22 * np.abs(u)
            du += 2.0 ** -39 * (self.K / 256 + 2) * absu.max(axis=1, keepdims=True)
            ref[at] += s * (u @ B.T)
            tol[at] += abs(s) * ((du + (r / 8 + 11) * 2 * EPS * np.abs(u)) @ np.abs(B).T)
        assert np.abs(ref).max() < 60000
        got = f64(out)
        assert not np.isnan(got).any()
        over = np.abs(got - ref) - (tol + 2.0 ** -11 * np.abs(ref))
        assert (over <= 0).all(), f"{np.abs(got - ref).max():.3e} off; {over.max():.3e} over what is allowed"


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("power", [-20, -17, -10])
def test_small_products_with_a_large_scale(shape, power):
    b = Batch(shape, scale=2.0 ** -power)
    b.run_and_check((b.randn(b.T, b.K) * 2.0 ** power).to(HF))


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_small_adapters(shape):
    """The smallness lies in A, and B is large."""
    b = Batch(shape, a_std=2.0 ** -16, b_std=2.0 ** 8, scale=-2.0 ** 9)
    b.run_and_check(b.randn(b.T, b.K).to(HF))


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_products_above_the_largest_fp16(shape):
    b = Batch(shape, a_std=2.0 ** 8, scale=2.0 ** -14)
    x = (b.randn(b.T, b.K) * 2.0 ** 10).to(HF)
    b.run_and_check(x, base=b.randn(b.T, b.N).to(HF))


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_rows_of_different_sizes(shape):
    """Each row has its own power of two, rows of zeros among them."""
    b = Batch(shape, scale=32.0)
    power = torch.randint(-20, 9, (b.T, 1), generator=b.gen, device="cuda")
    x = (b.randn(b.T, b.K) * 2.0 ** power).to(HF)
    x[b.T // 2] = 0
    b.run_and_check(x)
    base = b.randn(b.T, b.N).to(HF)
    b.run_and_check(x, base=base)
    assert torch.equal(b.hm(x, b.ids, base=base)[b.T // 2], base[b.T // 2])


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_ranks_of_different_sizes(shape):
    """In one row, u falls by powers of two over the ranks, and B grows by the same."""
    b = Batch(shape, scale=2.0 ** 12, by_rank=True)
    b.run_and_check((b.randn(b.T, b.K) * 2.0 ** -8).to(HF))


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_an_infinite_product_beside_finite_ones(shape):
    """u = (+inf, -2e5): the result is B's first column times infinity, since -2e5 is not infinite."""
    T, K, N, slots, most = shape
    b = Batch(shape)
    A, B = torch.zeros((2, K), device="cuda"), torch.ones((N, 2), device="cuda")
    A[0, 0], A[1, 1] = float("inf"), -4.0
    B[1::2, 0] = -1.0
    for i in range(slots):
        b.hm.load(i, A.to(HF), B.to(HF), 1.0)
    x = torch.zeros((T, K), dtype=HF, device="cuda")
    x[:, 0], x[:, 1] = 1.0, 50000.0
    out = b.hm(x, b.ids)
    assert (out[:, 0::2] == float("inf")).all() and (out[:, 1::2] == -float("inf")).all()


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_a_scale_near_the_largest_float(shape):
    """A zero column of B stays the base however large the scale and u are; no product of theirs is formed alone."""
    T, K, N, slots, most = shape
    b = Batch(shape)
    A, B = torch.full((1, K), 1.0, device="cuda"), torch.zeros((N, 1), device="cuda")
    B[0] = 1.0
    for i in range(slots):
        b.hm.load(i, A.to(HF), B.to(HF), 2.0e38)
    x, base = torch.full((T, K), 30000.0, device="cuda").to(HF), b.randn(T, N).to(HF)
    out = b.hm(x, b.ids, base=base)
    assert (out[:, 0] == float("inf")).all() and torch.equal(out[:, 1:], base[:, 1:])
