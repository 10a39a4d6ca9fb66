"""Results of the whole layer for a few tokens over its input or over one another are refused."""

import pytest
import torch

import nf3_moe_gb300 as hm
from tests.test_gpu_decode import make

pytestmark = pytest.mark.gpu


def test_ids_and_gates_over_other_arguments():
    L, moe, x, router = make(2, 256, 128, 4, 2, kept=2)
    words = torch.zeros(1024, dtype=torch.int32, device="cuda")    # 2 x 256 16-bit values are 256 words
    rows = lambda at: words[at:at + 256].view(x.dtype).view(2, 256)  # noqa: E731
    ids = lambda at: words[at:at + 4].view(2, 2)  # noqa: E731
    gates = lambda at: words[at:at + 4].view(torch.float32).view(2, 2)  # noqa: E731
    rows(0).copy_(x)
    want = moe.decode(x, router)
    fits = dict(out=256, ids=512, gates=516)
    for kw in (dict(ids=0), dict(ids=255), dict(gates=100), dict(ids=256), dict(gates=511), dict(ids=509), dict(gates=512), dict(gates=515),
               dict(ids=516), dict(out=252), dict(out=508)):
        a = fits | kw
        with pytest.raises(hm.HmoeError, match="overlap") as ei:
            moe.decode(rows(0), router, out=rows(a["out"]), ids=ids(a["ids"]), gates=gates(a["gates"]))
        assert ei.value.status == -1
    got = moe.decode(rows(0), router, out=rows(256), ids=ids(512), gates=gates(516))
    assert all(torch.equal(p, q) for p, q in zip(got, want)) and torch.equal(rows(0), x)
