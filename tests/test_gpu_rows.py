"""GPU tests of the row dispatch, the combine and their gradients against the float64 oracle.

Tolerances. u is the row type's rounding unit (bf16 2^-8, fp16 2^-11, fp32 2^-24), e = 2^-24:
  a row or an output: u |ref| for the rounding, (topk + 2) e sum|terms| for the fp32 sum, 2^-25 for fp16 subnormals;
  a dot product over H: a lane sums at most H / 32 + 8 products and the lanes join in at most 13 more steps, so
  (H / 32 + 21) e sum|terms|;
  a logit's gradient: its formula with those errors, and (topk + 3) e of its terms.
"""

import numpy as np
import pytest
import torch

import nf3_moe_gb300 as hm
from oracle import rows as orows

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
ROW = {torch.bfloat16: hm.ROW_BF16, torch.float16: hm.ROW_F16, torch.float32: hm.ROW_F32}
BF, HF, FF = torch.bfloat16, torch.float16, torch.float32


def f64(t):
    return t.detach().double().cpu().numpy()


def ints(*shape, fill=-77):
    return torch.full(shape, fill, dtype=torch.int32, device="cuda")


class Case:
    """Routes, inputs and the buffers of every call, outputs filled with NaN (-77 for whole numbers) first."""

    def __init__(self, T, E, k, H, dt, align=1, capacity=0, seed=0, skew=0.0):
        g = torch.Generator(device="cuda").manual_seed(seed * 1000 + T + E)
        logits = torch.randn((T, E), generator=g, device="cuda") - skew * torch.arange(E, device="cuda")
        self.T, self.E, self.k, self.H, self.dt, self.align, self.capacity = T, E, k, H, dt, align, capacity
        self.logits = logits
        top, idx = torch.sort(logits, dim=1, descending=True, stable=True)
        self.ids = idx[:, :k].to(torch.int32).contiguous()
        self.gates = torch.softmax(top[:, :k], dim=1).contiguous()
        flat = self.ids.reshape(-1).long()
        self.perm = torch.sort(flat, stable=True)[1].to(torch.int32)
        self.offsets = torch.cat([flat.new_zeros(1), torch.bincount(flat, minlength=E).cumsum(0)]).to(torch.int32)
        self.desc = hm.DispatchDesc(H, E, k, ROW[dt], align, capacity)
        self.R = hm.hmoe_dispatch_rows(self.desc, T)
        self.ws = torch.zeros(hm.hmoe_dispatch_workspace_size(self.desc, T), dtype=torch.uint8, device="cuda")
        self.x = torch.randn((T, H), generator=g, device="cuda").to(dt)
        self.y = torch.randn((self.R, H), generator=g, device="cuda").to(dt)
        self.maps = orows.row_maps(self.ids.cpu().numpy(), E, align, capacity)
        self.row_slot = torch.tensor(self.maps[0], dtype=torch.int32, device="cuda")
        self.slot_row = torch.tensor(self.maps[1], dtype=torch.int32, device="cuda").reshape(T, k)

    def wide(self, n):
        return torch.full((n, self.H), float("nan"), dtype=self.dt, device="cuda")

    def dispatch(self, gates=None, x=None, perm=None, offsets=None):
        out = self.wide(self.R), ints(self.R), ints(self.T, self.k), ints(self.E + 1)
        hm.hmoe_dispatch(self.desc, self.x if x is None else x, self.perm if perm is None else perm,
                         self.offsets if offsets is None else offsets, *out, self.ws, gates=gates)
        return out

    def combine(self, gates=None, y=None):
        out = self.wide(self.T)
        hm.hmoe_combine(self.desc, self.y if y is None else y, self.slot_row, out, self.ws, gates=gates)
        return out

    def grads(self):
        return torch.full((self.T, self.k), float("nan"), device="cuda"), torch.full((self.T, self.E), float("nan"), device="cuda")

    def ok(self):
        hm.hmoe_check_device_status(self.ws)


def close(got, ref, tol, what):
    got = f64(got)
    assert got.shape == ref.shape
    assert not np.isnan(got).any(), f"{what}: NaN (or unwritten)"
    over = np.abs(got - ref) - tol
    assert (over <= 0).all(), f"{what}: {np.abs(got - ref).max():.3e} off, allowed {tol.flat[over.argmax()]:.3e} there"


def rounding(dt, ref):
    return UNIT[dt] * np.abs(ref) + (2.0 ** -25 if dt == HF else 0.0)


def check_gate_grads(c, rows, v, dgates, dlogits):
    ids, gates = c.ids.cpu().numpy(), f64(c.gates)
    dg, size = orows.gate_grads(f64(rows), f64(v), c.maps[1])
    e_dg = (c.H / 32 + 21) * EPS * size
    close(dgates, dg, e_dg, "dgates")
    dl = orows.logit_grads(dg, gates, ids, c.E)
    e_dl = np.zeros_like(dl)
    for t in range(c.T):
        shared = float(np.dot(gates[t], e_dg[t] + (c.k + 3) * EPS * np.abs(dg[t])))
        for j in range(c.k):
            e_dl[t, ids[t, j]] = gates[t, j] * (e_dg[t, j] + shared + 3 * EPS * np.abs(dg[t, j]))
    close(dlogits, dl, e_dl, "dlogits")


SHAPES = [  # T, E, k, H, dtype, align, capacity
    (1, 1, 1, 1, FF, 1, 0), (1, 8, 2, 64, BF, 1, 0), (3, 4, 4, 7, HF, 1, 0), (8, 256, 8, 256, BF, 1, 0), (37, 8, 2, 256, BF, 1, 0),
    (37, 8, 2, 256, HF, 16, 0), (64, 16, 3, 1001, FF, 1, 0), (65, 16, 5, 1000, BF, 128, 9), (29, 512, 32, 72, HF, 1, 0),
    (130, 128, 9, 136, FF, 8, 4), (257, 5, 1, 2048, BF, 1, 0), (200, 3, 2, 520, HF, 1, 1), (19, 8, 2, 6144, BF, 1024, 0),
    (33, 7, 7, 33, BF, 3, 20), (513, 32, 4, 24, FF, 1, 0), (2, 300, 16, 2056, HF, 64, 0),
    # many tokens of narrow rows: 32 to 128 threads a token, and a last CTA that is not full
    (701, 16, 4, 256, BF, 1, 0), (613, 8, 2, 64, HF, 1, 0), (650, 12, 3, 200, FF, 16, 0), (903, 32, 9, 1000, BF, 8, 0),
    (643, 6, 2, 1536, HF, 1, 0), (700, 64, 32, 33, BF, 1, 0), (777, 5, 2, 130, FF, 1, 0), (1001, 20, 3, 712, FF, 1, 0),
    (811, 8, 2, 328, HF, 32, 150), (621, 4, 1, 24, BF, 1, 100), (2051, 8, 8, 8, HF, 4, 2000), (610, 3, 3, 1, BF, 1, 0),
    # odd widths below, at and past what a CTA's threads take together
    (9, 64, 8, 6001, BF, 1, 0), (3, 4, 2, 4099, FF, 1, 0), (700, 5, 2, 1025, HF, 16, 0), (6, 9, 3, 1023, BF, 1, 1)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("weighted", [False, True])
def test_dispatch_and_combine(shape, weighted):
    c = Case(*shape)
    gates = c.gates if weighted else None
    rows, row_slot, slot_row, row_offsets = c.dispatch(gates)
    assert np.array_equal(row_slot.cpu().numpy(), c.maps[0])
    assert np.array_equal(slot_row.cpu().numpy(), c.maps[1])
    assert np.array_equal(row_offsets.cpu().numpy(), c.maps[2])
    ref = orows.dispatch(f64(c.x), c.maps[0], c.k, f64(c.gates) if weighted else None)
    if weighted:
        close(rows, ref, rounding(c.dt, ref) + EPS * np.abs(ref), "rows")
    else:
        assert np.array_equal(f64(rows), ref)
    out = c.combine(gates)
    g64 = f64(c.gates) if weighted else None
    ref = orows.combine(f64(c.y), c.maps[1], g64)
    close(out, ref, rounding(c.dt, ref) + (c.k + 2) * EPS * orows.combine(np.abs(f64(c.y)), c.maps[1], g64), "out")
    c.ok()


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("weighted", [False, True])
def test_gradients(shape, weighted):
    c = Case(*shape, seed=1)
    gates = c.gates if weighted else None
    g64 = f64(c.gates) if weighted else None
    more, dgates, dlogits = {}, *c.grads()
    if weighted:
        more = dict(gates=gates, ids=c.ids, dgates=dgates, dlogits=dlogits)
    dx = c.wide(c.T)
    hm.hmoe_dispatch_backward(c.desc, c.y, c.slot_row, dx, c.ws, x=c.x if weighted else None, **more)
    ref = orows.combine(f64(c.y), c.maps[1], g64)
    close(dx, ref, rounding(c.dt, ref) + (c.k + 2) * EPS * orows.combine(np.abs(f64(c.y)), c.maps[1], g64), "dx")
    if weighted:
        check_gate_grads(c, c.y, c.x, dgates, dlogits)
        dgates.fill_(float("nan"))
        dlogits.fill_(float("nan"))
    drows = c.wide(c.R)
    hm.hmoe_combine_backward(c.desc, c.x, c.row_slot, c.slot_row, drows, c.ws, rows=c.y if weighted else None, **more)
    ref = orows.dispatch(f64(c.x), c.maps[0], c.k, g64)
    close(drows, ref, rounding(c.dt, ref) + EPS * np.abs(ref), "drows")
    if weighted:
        check_gate_grads(c, c.y, c.x, dgates, dlogits)
    c.ok()


@pytest.mark.parametrize("want", ["dgates", "dlogits", "none"])
def test_one_gate_gradient_alone(want):
    c = Case(21, 8, 2, 264, BF)
    both = dict(zip(("dgates", "dlogits"), c.grads()))
    hm.hmoe_combine_backward(c.desc, c.x, c.row_slot, c.slot_row, c.wide(c.R), c.ws, rows=c.y, gates=c.gates, ids=c.ids, **both)
    got = {want: torch.full_like(both[want], float("nan"))} if want != "none" else {}
    rows = c.wide(c.R)
    hm.hmoe_combine_backward(c.desc, c.x, c.row_slot, c.slot_row, rows, c.ws, rows=c.y, gates=c.gates, ids=c.ids, **got)
    if got:
        assert torch.equal(got[want], both[want])
    assert not rows.isnan().any()


def test_nothing_of_a_row_without_a_slot_reaches_a_result():
    """Pad rows of NaN and infinity, and a token whose every slot the capacity dropped."""
    c = Case(40, 4, 2, 128, BF, align=16, capacity=3, skew=2.0)
    pad = torch.tensor(c.maps[0] < 0, device="cuda")
    y = c.y.clone()
    y[pad] = float("nan")
    y[pad.nonzero()[::2, 0]] = float("inf")
    out = c.combine(c.gates, y)
    ref = orows.combine(f64(c.y), c.maps[1], f64(c.gates))
    close(out, ref, rounding(BF, ref) + 4 * EPS * orows.combine(np.abs(f64(c.y)), c.maps[1], f64(c.gates)), "out")
    empty = (c.maps[1] < 0).all(axis=1)
    assert empty.any() and not empty.all()
    assert (f64(out)[empty] == 0).all()
    dgates, dlogits = c.grads()
    hm.hmoe_dispatch_backward(c.desc, y, c.slot_row, c.wide(c.T), c.ws, x=c.x, gates=c.gates, ids=c.ids, dgates=dgates, dlogits=dlogits)
    check_gate_grads(c, c.y, c.x, dgates, dlogits)
    hm.hmoe_combine_backward(c.desc, c.x, c.row_slot, c.slot_row, c.wide(c.R), c.ws, rows=y, gates=c.gates, ids=c.ids, dgates=dgates,
                             dlogits=dlogits)
    check_gate_grads(c, c.y, c.x, dgates, dlogits)
    # a token of NaN marks its own rows only
    x = c.x.clone()
    x[5] = float("nan")
    rows = c.dispatch(x=x)[0]
    mine = torch.tensor((c.maps[0] >= 0) & (c.maps[0] // c.k == 5), device="cuda")
    assert torch.equal(rows.isnan().any(dim=1), mine)


@pytest.mark.parametrize("dt", [BF, HF, FF])
@pytest.mark.parametrize("H", [64, 65])
def test_tensors_off_the_vector_alignment(dt, H):
    """Contiguous tensors that start one element into their storage give the same bits."""
    c = Case(23, 8, 2, H, dt, align=4)
    off = lambda t: torch.cat([t.new_zeros(1), t.reshape(-1)])[1:].reshape(t.shape)  # noqa: E731
    a = c.dispatch(c.gates)
    x = off(c.x)
    assert x.data_ptr() % 16 != 0 and x.is_contiguous()
    b = c.dispatch(c.gates, x=x)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    assert torch.equal(c.combine(c.gates), c.combine(c.gates, off(c.y)))


def test_gradients_against_differences_of_the_calls():
    """The dispatch and the combine are linear in x, the rows and the gates: the change of the weighted output along a
    direction is the gradient's product with it (fp32 rows; errors of both sides by the sums' bounds)."""
    c = Case(31, 8, 3, 48, FF, align=4, capacity=10)
    er = hm.ExpertRows(c.H, c.E, c.k, dtype=FF, align=4, capacity=10)
    w = torch.randn((c.T, c.H), generator=torch.Generator(device="cuda").manual_seed(5), device="cuda")

    def through(x, gates):
        rows, plan = er.dispatch(x, c.perm, c.offsets)
        return er.combine(rows, plan, gates)

    x, gates = c.x.clone().requires_grad_(), c.gates.clone().requires_grad_()
    out = through(x, gates)
    out.backward(w)
    size = float((out.detach().abs().double() * w.abs().double()).sum())
    for v, grad, call in ((c.x, x.grad, lambda d: through(c.x + d, c.gates)), (c.gates, gates.grad, lambda d: through(c.x, c.gates + d))):
        d = torch.randn(v.shape, generator=torch.Generator(device="cuda").manual_seed(6), device="cuda")
        change = float(((call(d).double() - call(-d).double()) * w.double()).sum() / 2)
        want = float((grad.double() * d.double()).sum())
        far = float((call(d).abs().double() * w.abs().double()).sum()) + size + float((grad.abs() * d.abs()).double().sum())
        assert abs(change - want) <= (c.H / 32 + 30) * EPS * far


def test_autograd_of_the_router_and_both_sides():
    """A step through dispatch (gates at the rows) or combine (gates at the sum), bf16: the gradients that autograd
    hands out are the calls' own, and the logits' is the softmax formula's."""
    c = Case(50, 8, 2, 256, BF, align=16)
    er = hm.ExpertRows(c.H, c.E, c.k, dtype=BF, align=16)
    dout = torch.randn((c.T, c.H), device="cuda").to(BF)
    for at in ("combine", "dispatch"):
        x, logits = c.x.clone().requires_grad_(), c.logits.clone().requires_grad_()
        kw = dict(gates=c.gates, ids=c.ids, logits=logits)
        rows, plan = er.dispatch(x, c.perm, c.offsets, **(kw if at == "dispatch" else {}))
        assert torch.equal(plan.slot_row, c.slot_row)
        y = rows * 2
        y.retain_grad()
        out = er.combine(y, plan, **(kw if at == "combine" else {}))
        out.backward(dout)
        dgates, dlogits = c.grads()
        if at == "combine":
            drows = c.wide(c.R)
            hm.hmoe_combine_backward(c.desc, dout, c.row_slot, c.slot_row, drows, c.ws, rows=y.detach(), gates=c.gates, ids=c.ids,
                                     dgates=dgates, dlogits=dlogits)
            assert torch.equal(y.grad, drows)
        else:
            dx = c.wide(c.T)
            hm.hmoe_dispatch_backward(c.desc, (y.grad * 2), c.slot_row, dx, c.ws, x=c.x, gates=c.gates, ids=c.ids, dgates=dgates,
                                      dlogits=dlogits)
            assert torch.equal(x.grad, dx)
        assert torch.equal(logits.grad, dlogits)
    hm.hmoe_check_device_status(er.ws)


@pytest.mark.parametrize("what", ["perm", "offsets", "slot_row", "ids"])
def test_bad_routes_are_skipped_and_reported(what):
    c = Case(37, 8, 2, 256, BF)
    if what == "perm":
        bad = c.perm.clone()
        bad[3], bad[5] = 10_000, -4
        c.dispatch(perm=bad)
    elif what == "offsets":
        for i, v in ((8, 9_999), (0, -3), (4, 2_000_000_000), (2, 70)):
            bad = c.offsets.clone()
            bad[i] = v
            c.dispatch(offsets=bad)
            with pytest.raises(hm.HmoeError) as ei:
                c.ok()
            assert ei.value.status == -7
        bad = c.offsets.clone()
        bad[1:] = 2_147_483_647
        c.dispatch(offsets=bad)
    elif what == "slot_row":
        c.slot_row[2, 1] = c.R
        c.slot_row[3, 0] = 2_000_000_000
        c.combine(c.gates)
    else:
        ids = c.ids.clone()
        ids[7, 1] = 8
        dgates, dlogits = c.grads()
        hm.hmoe_combine_backward(c.desc, c.x, c.row_slot, c.slot_row, c.wide(c.R), c.ws, rows=c.y, gates=c.gates, ids=ids, dgates=dgates,
                                 dlogits=dlogits)
    with pytest.raises(hm.HmoeError) as ei:
        c.ok()
    assert ei.value.status == -7
    good = Case(37, 8, 2, 256, BF)                  # the context and the library still work
    assert torch.equal(good.dispatch()[0], good.dispatch()[0])
    good.ok()


def test_other_streams_graphs_and_repeats():
    c = Case(45, 16, 4, 512, BF, align=8)
    dgates, dlogits = c.grads()
    rows, row_slot, slot_row, row_offsets = (c.wide(c.R), ints(c.R), ints(c.T, c.k), ints(c.E + 1))
    out, drows = c.wide(c.T), c.wide(c.R)

    def step():
        hm.hmoe_dispatch(c.desc, c.x, c.perm, c.offsets, rows, row_slot, slot_row, row_offsets, c.ws)
        hm.hmoe_combine(c.desc, rows, slot_row, out, c.ws, gates=c.gates)
        hm.hmoe_combine_backward(c.desc, out, row_slot, slot_row, drows, c.ws, rows=rows, gates=c.gates, ids=c.ids, dgates=dgates,
                                 dlogits=dlogits)

    step()
    torch.cuda.synchronize()
    all_of = (rows, row_slot, slot_row, row_offsets, out, drows, dgates, dlogits)
    first = [t.clone() for t in all_of]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for t in all_of:
            t.zero_()
        step()
        graph = torch.cuda.CUDAGraph()
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, all_of))
        with torch.cuda.graph(graph, stream=side):
            step()
    for t in all_of:
        t.zero_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, all_of))


def test_no_write_outside_the_outputs():
    c = Case(27, 8, 2, 264, BF, align=4)
    def banded(*shape, dt):
        n = int(np.prod(shape))
        whole = torch.full((n + 512,), 3, dtype=dt, device="cuda")
        return whole, whole[256:256 + n].reshape(shape)
    bands = {"rows": banded(c.R, c.H, dt=BF), "row_slot": banded(c.R, dt=torch.int32), "slot_row": banded(c.T, c.k, dt=torch.int32),
             "row_offsets": banded(c.E + 1, dt=torch.int32), "out": banded(c.T, c.H, dt=BF), "drows": banded(c.R, c.H, dt=BF),
             "dgates": banded(c.T, c.k, dt=FF), "dlogits": banded(c.T, c.E, dt=FF)}
    b = {k: v[1] for k, v in bands.items()}
    hm.hmoe_dispatch(c.desc, c.x, c.perm, c.offsets, b["rows"], b["row_slot"], b["slot_row"], b["row_offsets"], c.ws)
    hm.hmoe_combine(c.desc, b["rows"], b["slot_row"], b["out"], c.ws, gates=c.gates)
    hm.hmoe_combine_backward(c.desc, b["out"], b["row_slot"], b["slot_row"], b["drows"], c.ws, rows=b["rows"], gates=c.gates, ids=c.ids,
                             dgates=b["dgates"], dlogits=b["dlogits"])
    for name, (whole, mid) in bands.items():
        n = mid.numel()
        assert (whole[:256] == 3).all() and (whole[256 + n:] == 3).all(), name


def test_empty_batch():
    c = Case(0, 8, 2, 64, BF, align=16)
    assert c.R == 0
    off = c.dispatch(c.gates)[3]
    assert (off == 0).all()
    assert c.combine().shape == (0, 64)
    c.ok()
