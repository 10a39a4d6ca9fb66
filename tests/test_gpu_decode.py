"""The whole layer for a few tokens (hmoe_decode) against its float64 oracle.

Tolerances: the oracle's bound on fp32 sums and on h as two values of the activation type, plus half a step of
the result's type (2^-8 of the value in bf16, 2^-11 in fp16). Gates: 1e-6, as for the routing.
"""

import numpy as np
import pytest
import torch

import nf3_moe_gb300 as hm
import synth
from oracle import decode as odec
from tests import gpu_util as U

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def make(T, H, I, E, k, kept_format=synth.FMT_NVFP4, kept=None, act="bf16", seed=0, max_tokens=8):
    """kept: experts of the kept tier (None: no bit map)."""
    L = synth.make_layer(H=H, I=I, E=E, topk=k, kept_ids=None if kept is None else list(range(0, E, max(1, E // max(1, kept))))[:kept],
                         uniform=kept is None, kept_format=kept_format, seed=seed, device="cuda", act=act)
    moe = U.build(L, max_tokens)
    gen = torch.Generator(device="cuda").manual_seed(seed * 31 + T)
    dt = moe.dtype
    x = torch.randn((T, H), generator=gen, device="cuda").to(dt)
    router = (torch.randn((E, H), generator=gen, device="cuda") * H ** -0.5).to(dt)
    return L, moe, x, router


def check(L, moe, x, router, got, bias=None, rows=None):
    out, ids, gates = got
    torch.cuda.synchronize()
    hm.hmoe_check_device_status(moe.decode_ws)
    b = None if bias is None else f64(bias)
    want_ids, want_gates = odec.route_of(f64(x), f64(router), L.topk, b)
    rows = list(range(x.shape[0])) if rows is None else rows
    assert np.array_equal(ids.cpu().numpy()[rows], want_ids[rows])
    assert np.abs(f64(gates)[rows] - want_gates[rows]).max() <= 1e-6
    ref, off = odec.forward(f64(x)[rows], want_ids[rows], want_gates[rows], L.expert_numpy, L.H, L.I, L.act)
    # half a step of fp16's subnormals; fp32 below its normal range, where h and each of the I products of a sum (of weights
    # below one) may lose up to 2^-126, in all k slots, whose gates sum to one
    tiny = 2.0 ** -25 if L.act == "f16" else 2 * L.I * 2.0 ** -126
    err = np.abs(f64(out)[rows] - ref)
    assert (err <= HALF[L.act] * (np.abs(ref) + off) + off + tiny).all(), float((err - off - HALF[L.act] * np.abs(ref)).max())


CASES = [
    # T, H, I, E, k, kept format, kept experts, type
    (1, 128, 64, 1, 1, synth.FMT_NVFP4, None, "bf16"),            # one expert, one unit a share at most
    (8, 128, 64, 8, 8, synth.FMT_NVFP4, None, "bf16"),            # every token to every expert: groups of eight
    (8, 256, 128, 8, 2, synth.FMT_NVFP4, 4, "bf16"),
    (5, 256, 192, 6, 3, synth.FMT_MXFP4, 3, "f16"),               # odd k-blocks of W2
    (8, 384, 320, 16, 4, synth.FMT_NVFP4, 5, "bf16"),
    (3, 256, 128, 40, 32, synth.FMT_NVFP4, 20, "bf16"),           # the largest top-k
    (8, 128, 64, 40, 32, synth.FMT_MXFP4, 20, "f16"),             # 256 slots
    (7, 128, 704, 3, 2, synth.FMT_NVFP4, 0, "f16"),               # nothing kept
    (8, 128, 64, 512, 8, synth.FMT_NVFP4, 100, "bf16"),           # the most experts
    (2, 2048, 768, 24, 8, synth.FMT_NVFP4, None, "bf16"),
    (6, 1024, 512, 5, 1, synth.FMT_MXFP4, 2, "bf16"),
    (8, 8192, 64, 2, 1, synth.FMT_NVFP4, 1, "bf16"),              # activations that fit a few tokens at a time
    (6, 128, 4096, 2, 2, synth.FMT_NVFP4, 1, "f16"),
    (4, 640, 1088, 9, 5, synth.FMT_MXFP4, 0, "bf16"),
    # more work a CTA than the 8 warps of the small calls are taken for
    (8, 1024, 512, 40, 8, synth.FMT_NVFP4, 20, "bf16"),
    (8, 640, 576, 12, 12, synth.FMT_MXFP4, 6, "f16"),             # every token to every expert, odd k-blocks of W2
    (1, 4096, 1024, 10, 10, synth.FMT_NVFP4, 5, "bf16"),
    (7, 1152, 640, 33, 9, synth.FMT_MXFP4, 16, "bf16"),
    (8, 8192, 256, 16, 4, synth.FMT_NVFP4, 8, "f16"),
    (6, 128, 8192, 6, 6, synth.FMT_NVFP4, 3, "f16"),
    (8, 1024, 704, 40, 8, synth.FMT_NVFP4, 20, "bf16"),
    (8, 640, 832, 12, 12, synth.FMT_MXFP4, 6, "f16"),
    (1, 4096, 1216, 10, 10, synth.FMT_NVFP4, 5, "bf16"),
    (6, 128, 9792, 6, 6, synth.FMT_NVFP4, 3, "f16"),
    # the limits: activations of one token fill shared memory
    (3, 39680, 64, 2, 1, synth.FMT_NVFP4, 1, "bf16"),
    (3, 128, 19840, 2, 2, synth.FMT_MXFP4, 1, "f16"),
    (8, 39680, 320, 4, 2, synth.FMT_NVFP4, 2, "f16"),             # with 16 warps
]


@pytest.mark.parametrize("T,H,I,E,k,fmt,kept,act", CASES)
def test_against_the_oracle(T, H, I, E, k, fmt, kept, act):
    L, moe, x, router = make(T, H, I, E, k, fmt, kept, act)
    check(L, moe, x, router, moe.decode(x, router))
    bias = torch.randn(E, generator=torch.Generator(device="cuda").manual_seed(7), device="cuda")
    check(L, moe, x, router, moe.decode(x, router, bias=bias), bias)


@pytest.mark.parametrize("act", ["bf16", "f16"])
def test_every_token_count_in_one_workspace(act):
    L, moe, x, router = make(8, 256, 192, 12, 4, kept=6, act=act)
    for T in (8, 1, 7, 2, 6, 3, 5, 4, 8, 0, 1):
        out, ids, gates = moe.decode(x[:T], router)
        assert out.shape == (T, 256) and ids.shape == gates.shape == (T, 4)
        if T:
            check(L, moe, x[:T], router, (out, ids, gates))
    # the status word, the counters (64 + 256 ints) and the largest |h| (256) are back at zero: what a later call relies on
    counters = 256 + (64 + 256) * 4 + 1024
    assert int(moe.decode_ws[:counters].count_nonzero()) == 0


def test_same_bits_again_and_without_ids():
    L, moe, x, router = make(8, 512, 320, 20, 6, kept=9)
    a = moe.decode(x, router)
    for _ in range(5):
        b = moe.decode(x, router)
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    out = torch.empty_like(a[0])
    hm.hmoe_decode(moe.layer, x, router, out, moe.decode_ws)
    assert torch.equal(out, a[0])


def test_near_the_forward_of_the_same_routes():
    L, moe, x, router = make(8, 512, 256, 16, 4, kept=8)
    out, ids, _ = moe.decode(x, router)
    other = moe(x, (x.float() @ router.float().T).contiguous())
    assert float((out.float() - other.float()).abs().max()) <= 2e-2 * float(other.float().abs().max())


def test_equal_logits_go_to_the_lower_ids():
    L, moe, x, router = make(4, 256, 64, 64, 8)
    router[:] = router[0]
    out, ids, gates = moe.decode(x, router)
    assert torch.equal(ids, torch.arange(8, device="cuda", dtype=torch.int32).expand(4, 8))
    assert torch.equal(gates, torch.full((4, 8), 0.125, device="cuda"))
    check(L, moe, x, router, (out, ids, gates))
    router[40:] = 2 * router[0]                                    # two levels: by value, then by id
    check(L, moe, x, router, moe.decode(x, router))


def test_experts_at_minus_infinity_are_not_chosen():
    L, moe, x, router = make(5, 256, 64, 40, 8, kept=10)
    bias = torch.zeros(40, device="cuda")
    bias[::2] = float("-inf")
    got = moe.decode(x, router, bias=bias)
    assert bool((got[1] % 2 == 1).all())
    check(L, moe, x, router, got, bias)


@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_one_token_that_is_not_finite_leaves_the_others(act, value):
    L, moe, x, router = make(6, 256, 128, 6, 3, kept=3, act=act)   # few experts: the tokens share them
    x[2, 17] = value
    out, ids, gates = moe.decode(x, router)
    assert bool(out[2].isnan().any()) and bool(((ids >= 0) & (ids < 6)).all())
    keep = [0, 1, 3, 4, 5]
    clean = torch.nan_to_num(x, 0.0, 0.0, 0.0)
    check(L, moe, clean, router, (out, ids, gates), rows=keep)


def test_fp16_h_beyond_the_types_range():
    """Activations of a thousand and more make |h| exceed 65504; the result is brought back by W2's global scale."""
    L, moe, x, router = make(5, 256, 128, 4, 2, act="f16")
    for ex in L.experts:
        c13, s13, g13 = ex["w13"]
        c2, s2, g2 = ex["w2"]
        ex["w13"], ex["w2"] = (c13, s13, g13 * 400.0), (c2, s2, g2 * 1e-4)
    moe = U.build(L, 8)
    x = (x.float() * 50).half()
    ids, gates = odec.route_of(f64(x), f64(router), 2)
    big = []
    for t in range(5):
        w = odec.weights(L.expert_numpy(int(ids[t, 0]))["fmt"], *L.expert_numpy(int(ids[t, 0]))["w13"], 256)
        a = w @ f64(x)[t]
        big.append(np.abs(a[:128] / (1 + np.exp(-a[:128])) * a[128:]).max())
    assert max(big) > 65504
    check(L, moe, x, router, moe.decode(x, router))


def test_tiny_inputs():
    for act, scale in (("bf16", 2.0 ** -60), ("bf16", 2.0 ** -40), ("f16", 2.0 ** -12)):
        L, moe, x, router = make(3, 256, 128, 4, 2, kept=2, act=act)
        check(L, moe, x * scale, router, moe.decode(x * scale, router))
    L, moe, x, router = make(3, 256, 128, 4, 2, kept=2)
    out, _, _ = moe.decode(torch.zeros_like(x), router)
    assert not out.any()


def test_graph_and_other_streams():
    L, moe, x, router = make(4, 512, 256, 16, 4, kept=8)
    want = moe.decode(x, router)
    out, ids, gates = (torch.empty_like(t) for t in want)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        st.wait_stream(torch.cuda.default_stream())
        moe.decode(x, router, out=out, ids=ids, gates=gates)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            for _ in range(3):
                moe.decode(x, router, out=out, ids=ids, gates=gates)
    torch.cuda.synchronize()
    x2 = torch.randn(x.shape, generator=torch.Generator(device="cuda").manual_seed(5), device="cuda").to(x.dtype)
    for v in (x2, x.clone(), x2):
        x.copy_(v)
        g.replay()
        torch.cuda.synchronize()
        check(L, moe, x, router, (out, ids, gates))


def test_two_graphs_share_a_workspace():
    """Graphs of one layer with different numbers of tokens (and warps a CTA), replayed in turn on one stream."""
    L, moe, x, router = make(8, 1024, 512, 20, 8, kept=10, act="f16")
    big, small = [t.clone() for t in moe.decode(x, router)], [t.clone() for t in moe.decode(x[:1], router)]
    outs, graphs, st = [[torch.empty_like(t) for t in w] for w in (big, small)], [], torch.cuda.Stream()
    st.wait_stream(torch.cuda.default_stream())
    with torch.cuda.stream(st):
        for o, v in zip(outs, (x, x[:1])):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                moe.decode(v, router, out=o[0], ids=o[1], gates=o[2])
            graphs.append(g)
        for _ in range(3):
            for o, g, want in zip(outs, graphs, (big, small)):
                o[0].fill_(7.0)
                g.replay()
                g.replay()
                st.synchronize()
                assert all(torch.equal(p, q) for p, q in zip(o, want))
    hm.hmoe_check_device_status(moe.decode_ws)
    check(L, moe, x, router, big)


def test_two_layers_at_once():
    """Two calls that share the GPU: neither may wait for a place the other holds."""
    made = [make(8, 1024, 512, 16, 4, kept=8, seed=s) for s in (1, 2)]
    want = [moe.decode(x, router) for _, moe, x, router in made]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[torch.empty_like(t) for t in w] for w in want]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, (_, moe, x, router), o in zip(streams, made, outs):
            with torch.cuda.stream(st):
                moe.decode(x, router, out=o[0], ids=o[1], gates=o[2])
    torch.cuda.synchronize()
    for (_, moe, _, _), w, o in zip(made, want, outs):
        hm.hmoe_check_device_status(moe.decode_ws)
        assert all(torch.equal(p, q) for p, q in zip(w, o))


def test_nothing_beside_the_buffers_is_written():
    L, moe, x, router = make(3, 256, 128, 8, 2, kept=4)
    d = moe.desc
    n = hm.hmoe_decode_workspace_size(d, 3)
    buf = torch.full((n + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    ws = buf[256:256 + n]
    hm.hmoe_workspace_init(ws)
    out = torch.full((5, 256), 7.0, dtype=x.dtype, device="cuda")
    ids = torch.full((5, 2), -7, dtype=torch.int32, device="cuda")
    gates = torch.full((5, 2), -7.0, device="cuda")
    xs, rs = x.clone(), router.clone()
    hm.hmoe_decode(moe.layer, x, router, out[1:4], ws, ids=ids[1:4], gates=gates[1:4])
    torch.cuda.synchronize()
    hm.hmoe_check_device_status(ws)
    assert bool((buf[:256] == 0x5A).all()) and bool((buf[256 + n:] == 0x5A).all())
    for t, v in ((out, 7.0), (ids, -7), (gates, -7.0)):
        assert bool((t[0] == v).all()) and bool((t[4] == v).all())
    assert torch.equal(x, xs) and torch.equal(router, rs)


def test_a_wait_that_runs_out_is_reported():
    """The counter of claimed shares set as if every W13 share were taken: the shares of W2 then wait for units that
    nobody computes. They give up after their limit and report it, and a zeroed workspace works again."""
    L, moe, x, router = make(2, 256, 128, 4, 2, kept=2)
    shares = torch.cuda.get_device_properties(0).multi_processor_count
    moe.decode_ws[256:260] = torch.tensor([shares], dtype=torch.int32).view(torch.uint8).cuda()
    moe.decode(x, router)
    torch.cuda.synchronize()
    with pytest.raises(hm.HmoeError) as ei:
        hm.hmoe_check_device_status(moe.decode_ws)
    assert ei.value.status == -6
    hm.hmoe_workspace_init(moe.decode_ws)
    check(L, moe, x, router, moe.decode(x, router))


def test_results_over_x_are_refused():
    L, moe, x, router = make(2, 256, 128, 4, 2, kept=2)
    flat = torch.zeros(2 * 512, dtype=x.dtype, device="cuda")
    flat[256:768] = x.flatten()
    for lo in (0, 256, 264, 504):
        with pytest.raises(hm.HmoeError, match="overlap"):
            moe.decode(flat[256:768].view(2, 256), router, out=flat[lo:lo + 512].view(2, 256))
    token = torch.stack([x[0], x[0]])
    moe.decode(token[:1], router, out=token[1:])                   # beside it
    assert torch.equal(token[1:], moe.decode(x[:1], router)[0])


def test_refusals():
    L, moe, x, router = make(2, 256, 128, 4, 2, kept=2)
    with pytest.raises(hm.HmoeError) as ei:                        # more tokens than the entry point takes
        moe.decode(torch.zeros((9, 256), dtype=x.dtype, device="cuda"), router)
    assert ei.value.status == -2
    small = U.build(L, 1)
    with pytest.raises(hm.HmoeError) as ei:                        # more than the workspace was made for
        small.decode(x, router)
    assert ei.value.status == -3
    with pytest.raises(hm.HmoeError) as ei:
        moe.decode(x, router, out=x)
    assert ei.value.status == -1
    for H, I in ((39680 + 128, 64), (128, 19840 + 64)):            # activations of a token above shared memory
        with pytest.raises(hm.HmoeError) as ei:
            hm.hmoe_decode_workspace_size(hm.LayerDesc(H, I, 4, 2, hm.FMT_NVFP4), 1)
        assert ei.value.status == -2
    flat = torch.zeros(2 * 256 + 8, dtype=x.dtype, device="cuda")
    with pytest.raises(hm.HmoeError) as ei:
        moe.decode(flat[1:513].view(2, 256), router)
    assert ei.value.status == -1
    for bad in (x.half(), x.cpu(), x[:, :128], x.t()):
        with pytest.raises(ValueError):
            moe.decode(bad, router)
    with pytest.raises(ValueError):
        moe.decode(x, router[:3])
    for name in ("x", "router"):
        a = {"x": x, "router": router}
        a[name] = a[name].clone().requires_grad_()
        with pytest.raises(RuntimeError, match=name):
            moe.decode(**a)
        with torch.no_grad():
            moe.decode(**a)
    q = hm.HybridMoELayer(256, 128, 4, 2, [int(b) for b in L.bit_map], U.device_experts(L), max_tokens=2, act_globals=(1.0, 1.0))
    with pytest.raises(hm.HmoeError) as ei:                        # W4A4 layers
        q.decode(x, router)
    assert ei.value.status == -2
    # a write that autograd has to know of
    out = torch.zeros((2, 256), dtype=x.dtype, device="cuda")
    before = out._version
    moe.decode(x, router, out=out)
    assert out._version > before
