"""CPU tests of the row dispatch: sizes and refusals of the library, the binding's tensor checks, and the
oracle's own identities (the combine is the dispatch's transpose; gradients against differences)."""

import ctypes

import numpy as np
import pytest
import torch

import nf3_moe_gb300 as hm
from nf3_moe_gb300 import rows as rows_mod
from oracle import rows as orows


@pytest.fixture(scope="module")
def lib():
    import os
    from nf3_moe_gb300 import _lib, build
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return _lib.lib()


@pytest.mark.parametrize("T,topk,E,align,capacity", [(0, 2, 8, 1, 0), (1, 1, 1, 1, 0), (8, 8, 256, 1, 0), (5, 2, 8, 16, 0),
                                                     (37, 2, 8, 128, 3), (4096, 8, 256, 128, 160), (7, 3, 512, 1024, 1)])
def test_row_count_matches_the_oracle(lib, T, topk, E, align, capacity):
    d = hm.DispatchDesc(64, E, topk, hm.ROW_BF16, align, capacity)
    assert hm.hmoe_dispatch_rows(d, T) == orows.row_count(T, topk, E, align, capacity)


@pytest.mark.parametrize("seed", range(6))
def test_row_count_holds_every_route(seed):
    rng = np.random.default_rng(seed)
    for _ in range(20):
        E = int(rng.integers(1, 12))
        k = int(rng.integers(1, min(E, 4) + 1))
        T, align, cap = int(rng.integers(0, 20)), int(rng.integers(1, 9)), int(rng.integers(0, 5))
        ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]) if T else np.zeros((0, k), int)
        row_slot, slot_row, off = orows.row_maps(ids, E, align, cap)
        assert off[-1] <= len(row_slot)
        for s, r in enumerate(slot_row.reshape(-1)):
            assert r < 0 or row_slot[r] == s


@pytest.mark.parametrize("desc,status", [
    (dict(row_dtype=3), -1), (dict(row_dtype=-1), -1), (dict(H=0), -1), (dict(E=0), -1), (dict(topk=0), -1),
    (dict(align=0), -1), (dict(capacity=-1), -1), (dict(E=513), -2), (dict(topk=9), -2), (dict(E=64, topk=33), -2),
    (dict(H=(1 << 20) + 1), -2), (dict(align=1025), -2)])
def test_bad_descriptors_are_refused(lib, desc, status):
    f = dict(H=64, E=8, topk=2, row_dtype=0, align=1, capacity=0) | desc
    d = hm.DispatchDesc(f["H"], f["E"], f["topk"], f["row_dtype"], f["align"], f["capacity"])
    for call in (lambda: hm.hmoe_dispatch_rows(d, 4), lambda: hm.hmoe_dispatch_workspace_size(d, 4)):
        with pytest.raises(hm.HmoeError) as ei:
            call()
        assert ei.value.status == status


def test_row_index_is_32_bits(lib):
    d = hm.DispatchDesc(64, 8, 2, hm.ROW_BF16, 1, 0)
    assert hm.hmoe_dispatch_rows(d, (2**31 - 1) // 2) == 2**31 - 2
    for bad, T in ((d, 2**30), (hm.DispatchDesc(64, 512, 1, 0, 1024, 0), 2**31 - 1000)):
        with pytest.raises(hm.HmoeError) as ei:
            hm.hmoe_dispatch_rows(bad, T)
        assert ei.value.status == -2
    with pytest.raises(hm.HmoeError) as ei:
        hm.hmoe_dispatch_rows(d, -1)
    assert ei.value.status == -1


def test_calls_are_refused_before_anything_is_enqueued(lib):
    d = hm.DispatchDesc(64, 8, 2, hm.ROW_BF16, 1, 0)
    b, p, q = ctypes.byref(d), 4096, 4098     # never dereferenced: every call below is refused on the host
    assert lib.hmoe_dispatch(b, None, 4, None, p, p, p, p, p, p, p, 256, None) == -1
    assert lib.hmoe_dispatch(b, p, 4, None, p, p, p, p, p, None, p, 256, None) == -1
    assert lib.hmoe_dispatch(b, p, -1, None, p, p, p, p, p, p, p, 256, None) == -1
    assert lib.hmoe_dispatch(b, p + 1, 4, None, p, p, p, p, p, p, p, 256, None) == -1     # not on an element
    assert lib.hmoe_dispatch(b, p, 4, None, p, p, p, p, p, p, p + 128, 256, None) == -1   # workspace not on 256 bytes
    assert lib.hmoe_dispatch(b, p, 4, None, p, p, p, p, p, p, p, 128, None) == -3
    assert lib.hmoe_dispatch(None, p, 4, None, p, p, p, p, p, p, p, 256, None) == -1
    assert lib.hmoe_combine(b, p, 4, None, None, p, p, 256, None) == -1
    assert lib.hmoe_combine(b, p, 4, p, None, q + 1, p, 256, None) == -1
    assert lib.hmoe_combine(b, p, 4, p, None, p, None, 256, None) == -1
    assert lib.hmoe_dispatch_backward(b, p, 4, p, None, p, p, p, p, None, p, 256, None) == -1   # dgates without x
    assert b"need gates" in lib.hmoe_last_error()
    assert lib.hmoe_dispatch_backward(b, p, 4, p, p, None, p, p, p, None, p, 256, None) == -1   # dgates without gates
    assert lib.hmoe_dispatch_backward(b, p, 4, p, p, p, None, p, None, p, p, 256, None) == -1   # dlogits without ids
    assert lib.hmoe_combine_backward(b, p, 4, None, p, None, None, None, p, None, None, p, 256, None) == -1
    assert lib.hmoe_combine_backward(b, p, 4, p, p, None, p, p, p, p, None, p, 256, None) == -1  # dgates without rows


def _bufs(T=4, k=2, E=8, H=64, dt=torch.bfloat16):
    R, i32 = T * k, torch.int32
    return dict(x=torch.zeros(T, H, dtype=dt), perm=torch.zeros(R, dtype=i32), offsets=torch.zeros(E + 1, dtype=i32),
                rows=torch.zeros(R, H, dtype=dt), row_slot=torch.zeros(R, dtype=i32), slot_row=torch.zeros(T, k, dtype=i32),
                row_offsets=torch.zeros(E + 1, dtype=i32), ws=torch.zeros(256, dtype=torch.uint8), gates=torch.zeros(T, k))


def test_binding_checks_of_dispatch(lib):
    d = hm.DispatchDesc(64, 8, 2, hm.ROW_BF16, 1, 0)
    assert rows_mod._check_dispatch(d, **_bufs(), cuda=False)[0] == 4
    for name, bad in (("x", torch.zeros(4, 63, dtype=torch.bfloat16)), ("x", torch.zeros(4, 64, dtype=torch.float16)),
                      ("x", torch.zeros(64, 4, dtype=torch.bfloat16).t()), ("perm", torch.zeros(8, dtype=torch.int64)),
                      ("perm", torch.zeros(7, dtype=torch.int32)), ("offsets", torch.zeros(8, dtype=torch.int32)),
                      ("rows", torch.zeros(7, 64, dtype=torch.bfloat16)), ("rows", torch.zeros(8, 64)),
                      ("row_slot", torch.zeros(9, dtype=torch.int32)), ("slot_row", torch.zeros(8, dtype=torch.int32)),
                      ("row_offsets", torch.zeros(8, dtype=torch.int32)), ("gates", torch.zeros(4, 2, dtype=torch.float64))):
        with pytest.raises(ValueError):
            rows_mod._check_dispatch(d, **(_bufs() | {name: bad}), cuda=False)
    with pytest.raises(TypeError):
        rows_mod._check_dispatch(d, **(_bufs() | {"perm": [0] * 8}), cuda=False)
    with pytest.raises(ValueError):
        rows_mod._check_dispatch(d, **_bufs())                        # not CUDA tensors


def test_binding_checks_of_the_gradients(lib):
    d = hm.DispatchDesc(64, 8, 2, hm.ROW_BF16, 1, 0)
    b = _bufs()
    ids, dg, dl = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2), torch.zeros(4, 8)
    dev = b["x"].get_device()
    check = lambda **kw: rows_mod._check_gate_grads(d, 4, dev, "x", **({"dot": b["x"], "dot_shape": b["x"].shape, "gates": b["gates"],  # noqa: E731
                                                    "ids": ids, "dgates": dg, "dlogits": dl} | kw), cuda=False)
    check()
    check(dlogits=None, ids=None)
    for kw in (dict(gates=None), dict(dot=None), dict(ids=None), dict(dgates=torch.zeros(4, 3)), dict(dlogits=torch.zeros(4, 7)),
               dict(ids=torch.zeros(4, 2, dtype=torch.int64)), dict(dot=torch.zeros(4, 64))):
        with pytest.raises(ValueError):
            check(**kw)
    with pytest.raises(ValueError):
        rows_mod._check_collect(d, "rows", torch.zeros(9, 64, dtype=torch.bfloat16), b["slot_row"], "out", b["x"], b["ws"], None,
                                cuda=False)
    with pytest.raises(ValueError):
        hm.ExpertRows(64, 8, 2, dtype=torch.float64, device="cpu")


def test_oracle_transpose_and_differences():
    """<combine(y), v> = <y, its gradient> and the gates' and logits' gradients against central differences."""
    rng = np.random.default_rng(3)
    T, k, E, H = 6, 3, 5, 7
    logits = rng.standard_normal((T, E))
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :k]
    row_slot, slot_row, _ = orows.row_maps(ids, E, 4, 3)
    y, v = rng.standard_normal((len(row_slot), H)), rng.standard_normal((T, H))

    def gates_of(lg):
        z = np.exp(np.take_along_axis(lg, ids, 1))
        return z / z.sum(1, keepdims=True)

    def loss(gates):
        return float((orows.combine(y, slot_row, gates) * v).sum())

    g = gates_of(logits)
    assert abs(loss(g) - float((y * orows.dispatch(v, row_slot, k, g)).sum())) < 1e-12
    dg, _ = orows.gate_grads(y, v, slot_row)
    dl = orows.logit_grads(dg, g, ids, E)
    h = 1e-6
    for t in range(T):
        for j in range(k):
            up, dn = g.copy(), g.copy()
            up[t, j] += h
            dn[t, j] -= h
            assert abs((loss(up) - loss(dn)) / (2 * h) - dg[t, j]) < 1e-7
        for e in range(E):
            up, dn = logits.copy(), logits.copy()
            up[t, e] += h
            dn[t, e] -= h
            assert abs((loss(gates_of(up)) - loss(gates_of(dn))) / (2 * h) - dl[t, e]) < 1e-7
