"""Calls that start while the ones before still write what they read: the same bits as with the GPU waited for in between."""

import pytest
import torch

import nf3_moe_gb300 as hm
from tests.test_gpu_decode import make

pytestmark = pytest.mark.gpu


def _linear(H, act, g):
    dt = torch.bfloat16 if act == "bf16" else torch.float16
    codes = torch.randint(0, 256, (H, H // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = (H ** -0.5 / 4.6 * (0.5 + torch.rand((H, H // 64), generator=g, device="cuda"))).to(dt)
    return hm.LinearInt4(H, H, 64, codes, scales, act_dtype=hm.ACT_BF16 if act == "bf16" else hm.ACT_F16)


@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("T", [1, 5, 8])
def test_each_call_reads_what_the_last_wrote(T, act):
    H = 512
    _, moe, x, router = make(T, H, 256, 16, 4, kept=8, act=act)
    g = torch.Generator(device="cuda").manual_seed(T)
    first, last = _linear(H, act, g), _linear(H, act, g)
    a, b, c = (torch.empty_like(x) for _ in range(3))
    bias = torch.randn(16, generator=g, device="cuda")

    def steps(wait):
        """Ten rounds over the same three buffers, each from the last one's result."""
        a.copy_(x)
        for _ in range(10):
            for call in (lambda: first(a, out=b), lambda: moe.decode(b, router, bias=bias, out=c), lambda: last(c, out=a)):
                call()
                if wait:
                    torch.cuda.synchronize()
            a.mul_(100.0).clamp_(-3, 3)                            # the layer's weights are small
            if wait:
                torch.cuda.synchronize()
        return a, b, c
    want = [t.clone() for t in steps(True)]
    assert all(bool(t.isfinite().all()) and bool(t.any()) for t in want)
    for _ in range(5):
        assert all(torch.equal(p, q) for p, q in zip(steps(False), want))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            got = steps(False)
    for _ in range(5):
        for t in got:
            t.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
    hm.hmoe_check_device_status(moe.decode_ws)
