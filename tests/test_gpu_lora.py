"""GPU tests of the low-rank adapters against the float64 oracle.

Tolerance of an output (e = 2^-24, p the type's significant bits, r the rank): A x is summed in fp32 in chains of at
most K / 16 + 16 steps (each at most 2 e, a tensor core may truncate), then enters the second product with 2 p bits;
that product adds r / 8 + 8 such steps, the scale and the base 3 more, and the result is rounded once, 2^-p (and
2^-25 for fp16 subnormals).
"""

import numpy as np
import pytest
import torch

import nf3_moe_gb300 as hm
from oracle import lora as olora

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
BF, HF = torch.bfloat16, torch.float16
BITS = {BF: 8, HF: 11}
ACT = {BF: hm.ACT_BF16, HF: hm.ACT_F16}


def f64(t):
    return t.double().cpu().numpy()


class Set:
    """A set of adapters with ranks from 1 to max_rank (slot 0 the largest), loaded and as float64 copies."""

    def __init__(self, K, N, slots, max_rank, dt, max_tokens, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed + K + N)
        self.K, self.N, self.dt, self.gen = K, N, dt, g
        self.hm = hm.LoraAdapters(K, N, slots, max_rank, max_tokens=max_tokens, act_dtype=ACT[dt])
        self.hm.packed[1024:].fill_(0xFF)                # empty slots hold NaN patterns: nothing reads them
        if slots > 128:
            self.hm = hm.LoraAdapters(K, N, slots, max_rank, max_tokens=max_tokens, act_dtype=ACT[dt])
        self.of, self.dev = {}, {}
        for i in range(slots):
            self.put(i, max_rank if i == 0 else 1 + (7 * i * i + 3 * i) % max_rank, 0.25 * (1 + i % 5))

    def randn(self, *shape, std=1.0):
        return (std * torch.randn(shape, generator=self.gen, device="cuda")).to(self.dt)

    def put(self, slot, rank, scale):
        A, B = self.randn(rank, self.K, std=self.K ** -0.5), self.randn(self.N, rank, std=rank ** -0.5)
        self.hm.load(slot, A, B, scale)
        self.of[slot] = (f64(A), f64(B), scale)

    def check(self, out, x, ids, base=None):
        assert not out.isnan().any()
        ids = ids.cpu().numpy()
        x64 = f64(x)
        ref = olora.forward(x64, ids, self.of, None if base is None else f64(base), self.N)
        tol = 2.0 ** -BITS[self.dt] * np.abs(ref) + (2.0 ** -25 if self.dt == HF else 0.0)
        if base is not None:
            tol += 6 * EPS * np.abs(f64(base))
        for t, a in enumerate(ids):
            if int(a) in self.of:
                A, B, scale = self.of[int(a)]
                r = A.shape[0]
                absu = np.abs(A) @ np.abs(x64[t])
                du = (self.K / 16 + 16) * 2 * EPS * absu + 2.0 ** (-2 * BITS[self.dt]) * np.abs(A @ x64[t])
                tol[t] += abs(scale) * (np.abs(B) @ (du + (r / 8 + 11) * 2 * EPS * np.abs(A @ x64[t])))
        got = f64(out)
        over = np.abs(got - ref) - tol
        assert (over <= 0).all(), f"{np.abs(got - ref).max():.3e} off, allowed {tol.flat[over.argmax()]:.3e}"


def ids_of(pattern, T, slots, seed=0):
    g = torch.Generator().manual_seed(seed + T)
    if pattern == "mixed":            # single tokens of many requests, some without an adapter
        ids = torch.randint(-1, slots, (T,), generator=g)
    elif pattern == "one":
        ids = torch.full((T,), slots - 1)
    elif pattern == "requests":       # prompt chunks side by side
        ids = torch.sort(torch.randint(0, slots, (T,), generator=g))[0]
        ids[T // 2:T // 2 + 3] = -1
    else:
        ids = torch.full((T,), -1)
    return ids.to(torch.int32).cuda()


SHAPES = [  # T, K, N, slots, max_rank, dtype, pattern
    (1, 8, 8, 1, 1, BF, "one"), (1, 2048, 2048, 16, 16, BF, "one"), (1, 512, 768, 4, 128, HF, "one"), (2, 72, 136, 3, 5, HF, "mixed"),
    (7, 64, 64, 2, 16, BF, "mixed"), (8, 256, 1000, 8, 64, BF, "mixed"), (9, 1000, 256, 8, 33, HF, "one"), (33, 328, 520, 40, 100, BF, "mixed"),
    (64, 6144, 512, 64, 64, BF, "mixed"), (64, 512, 6144, 300, 20, HF, "mixed"), (100, 2056, 72, 6, 48, BF, "requests"),
    (129, 64, 200, 3, 17, HF, "requests"), (257, 704, 384, 5, 128, BF, "requests"), (300, 136, 1032, 512, 8, BF, "mixed"),
    (513, 1032, 520, 12, 112, HF, "requests"), (700, 256, 256, 2, 16, BF, "one"), (1111, 320, 456, 32, 48, HF, "mixed"),
    (2050, 72, 64, 7, 80, BF, "requests"), (65, 128, 128, 4, 8, BF, "none"), (600, 128, 128, 4, 8, HF, "none"),
    (1536, 264, 136, 20, 24, BF, "mixed"), (1537, 264, 136, 20, 24, HF, "mixed"), (1700, 8, 8, 2, 1, BF, "requests"),
    (1600, 1032, 264, 3, 128, HF, "requests"), (3000, 136, 1000, 512, 112, BF, "mixed"), (4100, 72, 72, 30, 70, HF, "requests"),
    (2000, 64, 64, 1, 16, BF, "one"), (1800, 128, 128, 4, 8, HF, "none"), (2500, 2056, 520, 5, 96, BF, "requests"),
    (2600, 264, 72, 3, 16, HF, "mixed"), (2300, 1032, 328, 6, 128, BF, "requests"), (5000, 72, 1032, 2, 33, HF, "requests"),
    (2200, 520, 136, 40, 80, BF, "requests"), (8200, 64, 64, 5, 48, BF, "requests"), (9001, 8, 16, 3, 5, HF, "mixed"),
    (2400, 128, 128, 4, 8, BF, "none")]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("based", [True, False])
def test_forward(shape, based):
    T, K, N, slots, rank, dt, pattern = shape
    s = Set(K, N, slots, rank, dt, T)
    x, ids = s.randn(T, K), ids_of(pattern, T, slots)
    base = s.randn(T, N) if based else None
    out = torch.full((T, N), float("nan"), dtype=dt, device="cuda")
    s.hm(x, ids, base=base, out=out)
    s.check(out, x, ids, base)
    hm.hmoe_check_device_status(s.hm.ws)


@pytest.mark.parametrize("T", [1, 5, 40, 300, 700, 2900])
@pytest.mark.parametrize("dt", [BF, HF])
def test_column_ranges_and_in_place(T, dt):
    """x, base and out as column ranges of wider tensors, and in place; what lies beside them stays."""
    s = Set(200, 328, 5, 24, dt, T)
    wide_x, wide = s.randn(T, 456), s.randn(T, 2000)
    x, base, ids = wide_x[:, 56:256], wide[:, 1000:1328], ids_of("mixed", T, 5)
    want = s.hm(x.contiguous(), ids, base=base.contiguous())
    s.check(want, x, ids, base)
    before = wide.clone()
    got = s.hm(x, ids, base=base, out=wide[:, 8:336])
    assert torch.equal(got, want)
    s.hm(x, ids, base=base, out=base)
    assert torch.equal(base, want)
    before[:, 8:336] = want
    before[:, 1000:1328] = want
    assert torch.equal(wide, before)


@pytest.mark.parametrize("T", [6, 90, 640, 2900])
def test_rows_do_not_touch_each_other(T):
    """A row of NaN or infinity marks itself alone; a row without an adapter is base whatever its x holds."""
    s = Set(136, 200, 4, 20, BF, T)
    x, base, ids = s.randn(T, 136), s.randn(T, 200), ids_of("requests", T, 4)
    ids[0], ids[1], ids[2] = 2, -1, 2
    want = s.hm(x, ids, base=base)
    bad = x.clone()
    bad[0, 7], bad[1], bad[T - 1, 3] = float("nan"), float("nan"), float("inf")
    ids[T - 1] = 1
    want = s.hm(x, ids, base=base)
    got = s.hm(bad, ids, base=base)
    assert got[0].isnan().all() and not torch.isfinite(got[T - 1]).any()
    assert torch.equal(got[1], base[1])
    assert torch.equal(got[2:T - 1], want[2:T - 1])


@pytest.mark.parametrize("T", [4, 400, 2900])
def test_slots_are_replaced_emptied_and_checked(T):
    s = Set(128, 192, 3, 40, BF, T)
    x, base = s.randn(T, 128), s.randn(T, 192)
    ids = torch.arange(T, device="cuda", dtype=torch.int32) % 3
    s.check(s.hm(x, ids, base=base), x, ids, base)
    s.put(1, 3, -2.0)                                   # another rank and a negative scale
    s.check(s.hm(x, ids, base=base), x, ids, base)
    s.hm.unload(2)
    del s.of[2]
    out = s.hm(x, ids, base=base)
    s.check(out, x, ids, base)
    assert torch.equal(out[2::3], base[2::3])
    bad = ids.clone()
    bad[1], bad[T - 1] = 3, -2
    out = s.hm(x, bad, base=base)
    with pytest.raises(hm.HmoeError) as ei:
        hm.hmoe_check_device_status(s.hm.ws)
    assert ei.value.status == -7
    assert torch.equal(out[1], base[1]) and torch.equal(out[T - 1], base[T - 1])
    s.check(out, x, bad, base)
    hm.hmoe_check_device_status(s.hm.ws)


def test_refusals_on_the_host():
    s = Set(64, 64, 2, 8, BF, 8)
    x, ids, out = s.randn(8, 64), ids_of("one", 8, 2), torch.zeros((8, 64), dtype=BF, device="cuda")
    h, ws = s.hm.lora, s.hm.ws
    with pytest.raises(hm.HmoeError) as ei:
        hm.hmoe_lora_forward(h, x, ids, out, ws[:256])
    assert ei.value.status == -3
    flat = torch.zeros(8 * 72 + 8, dtype=BF, device="cuda")
    for bad in (flat[1:513].reshape(8, 64), flat[:8 * 68].reshape(8, 68)[:, :64]):   # not on 16 bytes; a stride of 68
        with pytest.raises(hm.HmoeError) as ei:
            hm.hmoe_lora_forward(h, bad, ids, out, ws)
        assert ei.value.status == -1
    for slot, rank in ((2, 4), (-1, 4), (0, 9)):
        with pytest.raises(hm.HmoeError) as ei:
            hm.hmoe_lora_load(h, slot, s.randn(rank, 64), s.randn(64, rank))
        assert ei.value.status == -1
    with pytest.raises(hm.HmoeError) as ei:
        hm.hmoe_lora_load(h, 0, s.randn(4, 64), s.randn(64, 4), scale=float("nan"))
    assert ei.value.status == -1
    wide = torch.zeros((8, 128), dtype=BF, device="cuda")
    s.hm(x[:0], ids[:0], base=out[:0], out=out[:0])          # no rows: nothing to do
    hm.hmoe_lora_forward(h, x, ids, wide[:, :64], ws)


@pytest.mark.parametrize("T", [3, 64, 500, 2900])
def test_other_streams_graphs_and_repeats(T):
    s = Set(512, 640, 9, 32, BF, T)
    x, base, ids = s.randn(T, 512), s.randn(T, 640), ids_of("mixed", T, 9)
    want = s.hm(x, ids, base=base)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = torch.zeros_like(want)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            s.hm(x, ids, base=base, out=out)
        side.synchronize()
        assert torch.equal(out, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            s.hm(x, ids, base=base, out=out)
    # the graph reads ids and the slots anew
    ids.copy_(ids.flip(0))
    s.put(0, 7, 1.0)
    s.put(3, 30, 0.5)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    s.check(out, x, ids, base)
    assert torch.equal(out, s.hm(x, ids, base=base))


@pytest.mark.parametrize("T", [4, 70, 500, 2900])
def test_no_write_outside_out(T):
    s = Set(136, 72, 3, 9, HF, T)
    whole = torch.full((T * 72 + 512,), 3.0, dtype=HF, device="cuda")
    out = whole[256:256 + T * 72].reshape(T, 72)
    x, ids = s.randn(T, 136), ids_of("mixed", T, 3)
    s.hm(x, ids, out=out)
    s.check(out, x, ids)
    assert (whole[:256] == 3).all() and (whole[256 + T * 72:] == 3).all()


def test_workspace_serves_any_batch_up_to_its_size():
    s = Set(256, 256, 6, 32, BF, 2900)
    for T in (2900, 900, 1, 64, 513, 8, 2500, 899):
        x, base, ids = s.randn(T, 256), s.randn(T, 256), ids_of("mixed", T, 6)
        s.check(s.hm(x, ids, base=base), x, ids, base)


@pytest.mark.parametrize("shape", [(1500, 1032, 264, 3, 64, BF, "mixed"), (8200, 136, 72, 9, 16, HF, "mixed"), (20000, 72, 64, 4, 8, BF, "mixed")],
                         ids=str)
def test_the_same_inputs_give_the_same_bits(shape):
    """Groups of many tiles whose rows lie scattered, K shared by several CTAs: every pass sums in the same order."""
    T, K, N, slots, rank, dt, pattern = shape
    s = Set(K, N, slots, rank, dt, T)
    x, base, ids = s.randn(T, K), s.randn(T, N), ids_of(pattern, T, slots)
    first = s.hm(x, ids, base=base)
    s.check(first, x, ids, base)
    for _ in range(10):
        assert torch.equal(s.hm(x, ids, base=base), first)
