"""The 4-bit integer linear against its float64 oracle.

Tolerances: the oracle's bound on the fp32 sums, plus half a step of the result's type (2^-8 of the value in bf16,
2^-11 in fp16).
"""

import numpy as np
import pytest
import torch

import nf3_moe_gb300 as hm
from oracle import int4 as oint4

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
ACT = {"bf16": hm.ACT_BF16, "f16": hm.ACT_F16}
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def f64(t):
    return None if t is None else t.detach().float().cpu().numpy().astype(np.float64)


def make(T, N, K, group, act, zeros=False, bias=False, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 13 * T + N)
    dt = DT[act]
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = (0.005 * (0.5 + torch.rand((N, K // group), generator=g, device="cuda"))).to(dt)
    z = torch.randint(0, 16, (N, K // group), generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    b = torch.randn(N, generator=g, device="cuda").to(dt) if bias else None
    x = torch.randn((T, K), generator=g, device="cuda").to(dt)
    return hm.LinearInt4(N, K, group, codes, scales, z, act_dtype=ACT[act]), x, (codes, scales, z, b)


def check(out, x, made, group, act, rows=None):
    codes, scales, z, b = made
    rows = slice(None) if rows is None else rows
    args = (f64(x)[rows], codes.cpu().numpy(), f64(scales), None if z is None else z.cpu().numpy(), group, f64(b))
    ref, off = oint4.forward(*args), oint4.bound(*args, act=act)
    tiny = 2.0 ** -25 if act == "f16" else 0.0                    # half a step of fp16's subnormals
    err = np.abs(f64(out)[rows] - ref)
    assert (err <= HALF[act] * (np.abs(ref) + off) + off + tiny).all(), float((err - off - HALF[act] * np.abs(ref)).max())


@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,N,K", [(1, 1, 128), (1, 16, 256), (2, 17, 128), (3, 100, 640), (7, 33, 1152), (8, 48, 512), (9, 16, 128),
                                   (13, 250, 384), (16, 64, 2048), (17, 31, 256), (40, 40, 384)])
def test_against_the_oracle(T, N, K, group, act):
    for zeros, bias in ((False, False), (True, True)):
        linear, x, made = make(T, N, K, group, act, zeros, bias)
        check(linear(x, bias=made[3]), x, made, group, act)


@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("T,N,K,group", [(1, 40, 32, 32), (5, 20, 96, 32), (4, 64, 1056, 32), (2, 50, 192, 64), (3, 16, 4544, 64), (12, 30, 160, 32)])
def test_k_that_ends_inside_a_block(T, N, K, group, act):
    linear, x, made = make(T, N, K, group, act, True, True)
    check(linear(x, bias=made[3]), x, made, group, act)


@pytest.mark.parametrize("T,N,K,group,act", [(1, 6144, 6144, 128, "bf16"), (5, 4096, 6144, 64, "f16"), (16, 2048, 6144, 128, "bf16"),
                                             (8, 12000, 1024, 32, "bf16"), (2, 200, 32768, 128, "f16"), (9, 100, 16384, 64, "bf16"),
                                             # K in parts: many units a CTA, an uneven last part, a K of one row that does not fit
                                             (16, 40000, 4224, 128, "bf16"), (12, 3000, 6176, 32, "f16"), (1, 33, 131072, 128, "bf16"),
                                             (33, 64, 9216, 64, "bf16")])
def test_larger(T, N, K, group, act):
    linear, x, made = make(T, N, K, group, act, True, True)
    check(linear(x, bias=made[3]), x, made, group, act)


def test_column_ranges_and_one_row_of_any_stride():
    linear, x, made = make(6, 40, 256, 64, "bf16", True, True)
    wide, dest = torch.full((6, 600), 9.0, dtype=x.dtype, device="cuda"), torch.full((6, 100), 3.0, dtype=x.dtype, device="cuda")
    wide[:, 8:264] = x
    linear(wide[:, 8:264], bias=made[3], out=dest[:, 31:71])
    check(dest[:, 31:71], x, made, 64, "bf16")
    assert bool((dest[:, :31] == 3).all()) and bool((dest[:, 71:] == 3).all())
    assert torch.equal(linear(wide[2:3, 8:264], bias=made[3]), linear(x[2:3], bias=made[3]))


def test_rows_do_not_mix_and_zero_rows():
    for act in ("bf16", "f16"):
        linear, x, made = make(12, 50, 384, 128, act, True)
        assert linear(x[:0]).shape == (0, 50)
        clean = linear(x)
        for value in (float("nan"), float("inf")):
            y = x.clone()
            y[5, 100] = value
            out = linear(y)
            keep = [t for t in range(12) if t != 5]
            assert torch.equal(out[keep], clean[keep])
            assert not bool(out[5].isfinite().all())


def test_a_large_mean_of_x():
    """All of x alike: the offsets' share of the sums is as large as it gets."""
    for act in ("bf16", "f16"):
        linear, x, made = make(4, 64, 2048, 128, act, True)
        x = torch.full_like(x, 3.0) + 0.01 * x
        check(linear(x), x, made, 128, act)


def test_extremes_of_codes_zeros_and_scales():
    N, K, group = 32, 256, 64
    for act in ("bf16", "f16"):
        dt = DT[act]
        x = torch.randn((3, K), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(dt)
        scales = torch.tensor([2.0 ** -14, 1.0, 100.0, 0.0], device="cuda").to(dt).expand(N, 4).contiguous()
        for code, zero in ((0, 15), (255, 0), (255, 255), (0, 0)):
            codes = torch.full((N, K // 2), code, dtype=torch.uint8, device="cuda")
            z = torch.full((N, 4), zero, dtype=torch.uint8, device="cuda")  # the low four bits count
            out = hm.LinearInt4(N, K, group, codes, scales, z, act_dtype=ACT[act])(x)
            check(out, x, (codes, scales, z, None), group, act)


def test_same_bits_graph_and_streams():
    linear, x, made = make(4, 300, 1024, 128, "bf16", True, True)
    want = linear(x, bias=made[3])
    assert all(torch.equal(linear(x, bias=made[3]), want) for _ in range(5))
    out, st = torch.empty_like(want), torch.cuda.Stream()
    with torch.cuda.stream(st):
        st.wait_stream(torch.cuda.default_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            linear(x, bias=made[3], out=out)
    x2 = torch.randn_like(x)
    for v in (x2, x.clone()):
        x.copy_(v)
        g.replay()
        torch.cuda.synchronize()
        check(out, x, made, 128, "bf16")
    # one linear on two streams at once: it has no workspace
    outs, streams = [torch.empty_like(want) for _ in range(2)], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, o in zip(streams, outs):
            with torch.cuda.stream(s):
                linear(x, bias=made[3], out=o)
    torch.cuda.synchronize()
    assert all(torch.equal(o, linear(x, bias=made[3])) for o in outs)


def test_with_adapters():
    from oracle import lora as olora
    linear, x, made = make(6, 64, 256, 64, "bf16", True)
    adapters = hm.LoraAdapters(256, 64, slots=2, max_rank=8, max_tokens=6)
    A, B = (torch.randn((8, 256), device="cuda") / 16).bfloat16(), torch.randn((64, 8), device="cuda").bfloat16()
    adapters.load(1, A, B, 0.5)
    ids = torch.tensor([1, -1, 1, 0, 1, -1], dtype=torch.int32, device="cuda")
    base = linear(x)
    got = linear(x, adapters=adapters, ids=ids)
    ref = olora.forward(f64(x), ids.cpu().numpy(), {1: (f64(A), f64(B), 0.5)}, f64(base))
    size = olora.forward(np.abs(f64(x)), ids.cpu().numpy(), {1: (np.abs(f64(A)), np.abs(f64(B)), 0.5)}, np.abs(f64(base)))
    assert (np.abs(f64(got) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -15 * size).all()


def test_refusals():
    linear, x, made = make(3, 40, 256, 64, "bf16")
    flat = torch.zeros(3 * 256 + 8, dtype=x.dtype, device="cuda")
    with pytest.raises(hm.HmoeError) as ei:                        # x off its 16 bytes
        linear(flat[1:769].view(3, 256))
    assert ei.value.status == -1
    with pytest.raises(hm.HmoeError):
        linear(torch.zeros((3, 260), dtype=x.dtype, device="cuda")[:, :256])   # a row stride that is no multiple of 8
    for bad in (x.half(), x.cpu(), x[:, :128], x.t()):
        with pytest.raises(ValueError):
            linear(bad)
    with pytest.raises(ValueError):
        linear(x, bias=torch.zeros(41, dtype=x.dtype, device="cuda"))
    with pytest.raises(RuntimeError, match="gradient"):
        linear(x.clone().requires_grad_())
    with torch.no_grad():
        linear(x.clone().requires_grad_())
    out = torch.zeros((3, 40), dtype=x.dtype, device="cuda")
    before = out._version
    linear(x, out=out)
    assert out._version > before


def test_results_over_x_are_refused_and_beside_it_taken():
    linear, x, made = make(3, 40, 256, 64, "bf16")
    want, wide = linear(x), torch.zeros((3, 400), dtype=x.dtype, device="cuda")
    ranges = {lo: torch.as_strided(wide, (3, 40), (400, 1), lo) for lo in (0, 100, 217, 255, 256, 300, 360)}
    for lo in (0, 100, 217, 255):
        with pytest.raises(hm.HmoeError, match="overlap"):
            linear(wide[:, :256], out=ranges[lo])
    for lo in (256, 300, 360):                                     # columns behind x's
        wide[:, :256] = x
        linear(wide[:, :256], out=ranges[lo])
        assert torch.equal(ranges[lo], want) and torch.equal(wide[:, :256], x)
    wide.zero_()
    wide[:, 144:] = x                                              # columns before x's, and in the next row's end
    linear(wide[:, 144:], out=wide[:, 104:144])
    assert torch.equal(wide[:, 104:144], want)
    with pytest.raises(hm.HmoeError, match="overlap"):             # a row stride of its own over the same memory
        linear(wide[:, 144:], out=torch.as_strided(wide, (3, 40), (80, 1), 120))
    square, y, _ = make(1, 256, 256, 64, "f16")
    with pytest.raises(hm.HmoeError, match="overlap"):
        square(y, out=y)


def test_too_many_rows_are_refused():
    linear, x, _ = make(1, 16, 64, 64, "bf16")
    rows = (1 << 19) + 1
    many, out = x.new_zeros((rows, 64)), x.new_zeros((rows, 16))
    with pytest.raises(hm.HmoeError) as ei:
        linear(many, out=out)
    assert ei.value.status == -2
    many[-2] = x[0]
    assert torch.equal(linear(many[:-1])[-1:], linear(x)) and not bool(linear(many[:-1])[:-1].any())
