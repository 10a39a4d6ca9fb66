"""CPU tests of the rows' autograd: the library's calls are replaced by plain torch ones, the autograd code runs as it is."""

import pytest
import torch

import nf3_moe_gb300 as hm
from nf3_moe_gb300 import rows as rows_mod

T, E, K, H = 3, 4, 2, 8


def _dispatch_rows(desc, n):
    return n * desc.topk


def _dispatch(desc, x, perm, offsets, rows, row_slot, slot_row, row_offsets, ws, gates=None):
    slot = perm.long()
    g = 1.0 if gates is None else gates.reshape(-1)[slot][:, None]
    rows.copy_(x[slot // desc.topk] * g)
    row_slot.copy_(perm)
    flat = torch.empty_like(perm)
    flat[slot] = torch.arange(perm.numel(), dtype=torch.int32)
    slot_row.copy_(flat.reshape(slot_row.shape))
    row_offsets.copy_(offsets)


def _combine(desc, rows, slot_row, out, ws, gates=None):
    picked = rows[slot_row.long()]
    out.copy_((picked if gates is None else gates[:, :, None] * picked).sum(dim=1))


def _gate_grads(dot, gates, ids, dgates, dlogits):
    if dgates is not None:
        dgates.copy_(dot)
    if dlogits is not None:
        if ids is None:
            raise ValueError("dlogits needs ids")
        dlogits.zero_().scatter_(1, ids.long(), gates * (dot - (gates * dot).sum(dim=1, keepdim=True)))


def _dispatch_backward(desc, drows, slot_row, dx, ws, x=None, gates=None, ids=None, dgates=None, dlogits=None):
    _combine(desc, drows, slot_row, dx, ws, gates)
    if dgates is not None or dlogits is not None:
        _gate_grads((drows[slot_row.long()] * x[:, None]).sum(dim=2), gates, ids, dgates, dlogits)


def _combine_backward(desc, dout, row_slot, slot_row, drows, ws, rows=None, gates=None, ids=None, dgates=None, dlogits=None):
    slot = row_slot.long()
    drows.copy_(dout[slot // desc.topk] * (1.0 if gates is None else gates.reshape(-1)[slot][:, None]))
    if dgates is not None or dlogits is not None:
        _gate_grads((rows[slot_row.long()] * dout[:, None]).sum(dim=2), gates, ids, dgates, dlogits)


@pytest.fixture
def plain(monkeypatch):
    for name, call in (("hmoe_dispatch_rows", _dispatch_rows), ("hmoe_dispatch", _dispatch), ("hmoe_combine", _combine),
                       ("hmoe_dispatch_backward", _dispatch_backward), ("hmoe_combine_backward", _combine_backward)):
        monkeypatch.setattr(rows_mod, name, call)
    monkeypatch.setattr(rows_mod, "hmoe_dispatch_workspace_size", lambda desc, n: 256)
    torch.manual_seed(0)
    logits = torch.randn(T, E)
    top, ids = torch.sort(logits, dim=1, descending=True)
    ids = ids[:, :K].to(torch.int32).contiguous()
    flat = ids.reshape(-1).long()
    perm = torch.sort(flat, stable=True)[1].to(torch.int32)
    offsets = torch.cat([flat.new_zeros(1), torch.bincount(flat, minlength=E).cumsum(0)]).to(torch.int32)
    gates = torch.softmax(top[:, :K], dim=1).contiguous()
    er = hm.ExpertRows(H, E, K, dtype=torch.float32, device="cpu")
    return er, torch.randn(T, H), logits, ids, gates, perm, offsets


def test_first_derivatives(plain):
    """The replaced calls serve: gradients equal those of plain torch."""
    er, x, logits, ids, gates, perm, offsets = plain
    w = torch.randn(T, H)
    got, want = [], []
    for own in (True, False):
        xs, lg = x.clone().requires_grad_(), logits.clone().requires_grad_()
        if own:
            rows, plan = er.dispatch(xs, perm, offsets)
            out = er.combine(torch.sin(rows), plan, gates, ids=ids, logits=lg)
        else:
            g = torch.softmax(lg.gather(1, ids.long()), dim=1)
            out = (g[:, :, None] * torch.sin(xs)[:, None]).sum(dim=1)
        (got if own else want).extend(torch.autograd.grad((out * w).sum(), (xs, lg)))
    for a, b in zip(got, want):
        assert torch.allclose(a, b, atol=1e-6)


def _loss(plain, at, source, linear):
    """A loss through both calls; the gates are applied in `at`, and `source` (gates or logits) gets their gradient."""
    er, x, logits, ids, gates, perm, offsets = plain
    xs, gs, lg = x.clone().requires_grad_(), gates.clone(), logits.clone()
    kw = {"gates": gs}
    if source == "gates":
        gs.requires_grad_()
    elif source == "logits":
        lg.requires_grad_()
        kw.update(ids=ids, logits=lg)
    rows, plan = er.dispatch(xs, perm, offsets, **(kw if at == "dispatch" else {}))
    out = er.combine(rows * rows if at == "combine" else rows, plan, **(kw if at == "combine" else {}))
    return (out.sum() if linear else (out ** 2).sum()), xs, gs if source == "gates" else lg


@pytest.mark.parametrize("linear", [True, False])
@pytest.mark.parametrize("source", ["gates", "logits"])
@pytest.mark.parametrize("at", ["dispatch", "combine"])
def test_second_derivatives_are_refused(plain, at, source, linear):
    """A gradient that is used in a loss must not count as a constant: there is no second derivative, and that is said,
    whichever tensor is differentiated for, and where the incoming gradient is itself a constant too."""
    for way in ("backward", "of the source", "of x", "gradient of x"):
        loss, xs, src = _loss(plain, at, source, linear)
        (g,) = torch.autograd.grad(loss, xs if way == "gradient of x" else src, create_graph=True)
        assert g.requires_grad
        penalty = (g ** 2).sum() + loss
        with pytest.raises(RuntimeError, match="no second derivative"):
            if way == "backward":
                penalty.backward()
            else:
                torch.autograd.grad(penalty, xs if way == "of x" else src)


def test_a_constant_gradient_stays_one(plain):
    """Without gates to train, the gradient of a linear loss depends on nothing that requires one."""
    er, x, logits, ids, gates, perm, offsets = plain
    xs = x.clone().requires_grad_()
    rows, plan = er.dispatch(xs, perm, offsets)
    loss = er.combine(rows, plan, gates).sum()
    (g,) = torch.autograd.grad(loss, xs, create_graph=True)
    assert not g.requires_grad and torch.allclose(g, torch.ones_like(g))
    ((g ** 2).sum() * xs.sum() + er.combine(er.dispatch(xs, perm, offsets)[0], plan, gates).sum()).backward()
    assert torch.allclose(xs.grad, torch.full_like(g, float(T * H) + 1))


def test_create_graph_alone_changes_nothing(plain):
    loss, xs, src = _loss(plain, "combine", "logits", False)
    once = torch.autograd.grad(loss, (xs, src))
    loss, xs, src = _loss(plain, "combine", "logits", False)
    again = torch.autograd.grad(loss, (xs, src), create_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(once, again))


@pytest.mark.parametrize("at", ["dispatch", "combine"])
def test_logits_that_would_get_no_gradient_are_refused_at_once(plain, at):
    """Logits get theirs through the gates and the ids; where one is missing the call says so, not the backward (or
    nobody). Logits that want no gradient are no error."""
    er, x, logits, ids, gates, perm, offsets = plain
    rows, plan = er.dispatch(x, perm, offsets)

    def call(**kw):
        return er.dispatch(x, perm, offsets, **kw) if at == "dispatch" else er.combine(rows, plan, **kw)

    want = logits.clone().requires_grad_()
    for kw, missing in ((dict(gates=gates, logits=want), "ids"), (dict(ids=ids, logits=want), "gates"), (dict(logits=want), "gates")):
        with pytest.raises(ValueError, match=missing):
            call(**kw)
        with torch.no_grad():
            call(**kw)
        call(**(kw | {"logits": logits}))
    call(gates=gates, ids=ids, logits=want)
