"""Token rows sorted by expert and back, with the gates applied, and their gradients (include/hmoe.h).

The functions keep the C names and take torch tensors the caller owns. ``ExpertRows`` owns the
buffers instead and takes part in autograd:

    rows_of = ExpertRows(H, E, topk, max_tokens=T)
    ids, gates, perm, offsets = layer.plan(logits)
    rows, plan = rows_of.dispatch(x, perm, offsets)      # [R, H], each expert's rows side by side
    y = experts(rows, plan.row_offsets)                  # the caller's own work
    out = rows_of.combine(y, plan, gates, ids=ids, logits=logits)
    out.backward(...)                                    # x, y, gates and the router logits get gradients
"""

import ctypes
from typing import NamedTuple

import torch

from . import _lib, _need
from ._lib import ROW_BF16, ROW_F16, ROW_F32, DispatchDesc

_TORCH = {ROW_BF16: torch.bfloat16, ROW_F16: torch.float16, ROW_F32: torch.float32}
_ROW = {v: k for k, v in _TORCH.items()}
_INT_MAX = 2 ** 31 - 1  # of the library's int arguments; ctypes would pass the low 32 bits of more


def _int32(name, n):
    n = int(n)
    if not -_INT_MAX <= n <= _INT_MAX:
        raise ValueError(f"{name}={n} exceeds the library's 32-bit index")
    return n


def row_torch_dtype(row_dtype):
    """The torch dtype of rows for a ROW_* value."""
    return _TORCH[int(row_dtype)]


def _is(name, t, shape, dtype, device, cuda=True):
    """_need for a tensor that is nearly always right: one look, and the full check for its message. device: its
    index, as get_device gives it (-1 on the host)."""
    try:
        if t.shape == shape and t.dtype is dtype and t.is_contiguous() and (t.get_device() == device >= 0 or not cuda):
            return
    except AttributeError:
        pass
    _need(name, t, shape, dtype, device=torch.device("cuda", device) if device >= 0 else None, cuda=cuda)


def _is_ws(ws, device, cuda=True):
    try:
        if ws.is_contiguous() and (ws.get_device() == device >= 0 or not cuda):
            return
    except AttributeError:
        pass
    _need("ws", ws, device=torch.device("cuda", device) if device >= 0 else None, cuda=cuda)


def _raw(t):
    return None if t is None else t.data_ptr()


def _raw_stream(stream, device):
    """The stream's handle; None: the device's current stream (this look-up takes 0.1 us, the Stream object 2.9)."""
    return torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream


def _bytes(ws):
    return ws.nbytes


def hmoe_dispatch_rows(desc, T):
    """Rows of the sorted buffer for T tokens."""
    n = ctypes.c_int()
    _lib.check(_lib.lib().hmoe_dispatch_rows(ctypes.byref(desc), _int32("T", T), ctypes.byref(n)))
    return n.value


def hmoe_dispatch_workspace_size(desc, max_tokens):
    b = ctypes.c_size_t()
    _lib.check(_lib.lib().hmoe_dispatch_workspace_size(ctypes.byref(desc), _int32("max_tokens", max_tokens), ctypes.byref(b)))
    return b.value


def _check_tokens(name, desc, t, cuda):
    """T, H, the rows' dtype and the device index of a [T, H] tensor."""
    dt, H = _TORCH[desc.row_dtype], desc.H
    try:
        T, width = t.shape
        device = t.get_device()
        if width == H and t.dtype is dt and t.is_contiguous() and T <= _INT_MAX and (device >= 0 or not cuda):
            return T, H, dt, device
    except (AttributeError, ValueError):
        pass
    _need(name, t, (None, H), dt, cuda=cuda)
    return _int32(f"the rows of {name}", t.shape[0]), H, dt, t.get_device()


def _rows_of(desc, T):
    """hmoe_dispatch_rows, for a descriptor that the library's calls check."""
    slots, align, cap = T * desc.topk, desc.align, desc.capacity
    most = slots + min(desc.E, slots) * (align - 1)
    return min(most, -(-cap // align) * align * desc.E) if cap > 0 else most


def _check_dispatch(desc, x, perm, offsets, rows, row_slot, slot_row, row_offsets, ws, gates, cuda=True):
    T, H, dt, dev = _check_tokens("x", desc, x, cuda)
    R, k, E, i32 = _rows_of(desc, T), desc.topk, desc.E, torch.int32
    _is("perm", perm, (T * k,), i32, dev, cuda)
    _is("offsets", offsets, (E + 1,), i32, dev, cuda)
    _is("rows", rows, (R, H), dt, dev, cuda)
    _is("row_slot", row_slot, (R,), i32, dev, cuda)
    _is("slot_row", slot_row, (T, k), i32, dev, cuda)
    _is("row_offsets", row_offsets, (E + 1,), i32, dev, cuda)
    if gates is not None:
        _is("gates", gates, (T, k), torch.float32, dev, cuda)
    _is_ws(ws, dev, cuda)
    return T, dev


def _check_collect(desc, name, rows, slot_row, out_name, out, ws, gates, cuda=True):
    T, H, dt, dev = _check_tokens(out_name, desc, out, cuda)
    k = desc.topk
    _is(name, rows, (_rows_of(desc, T), H), dt, dev, cuda)
    _is("slot_row", slot_row, (T, k), torch.int32, dev, cuda)
    if gates is not None:
        _is("gates", gates, (T, k), torch.float32, dev, cuda)
    _is_ws(ws, dev, cuda)
    return T, dev


def _check_gate_grads(desc, T, dev, dot_name, dot, dot_shape, gates, ids, dgates, dlogits, cuda=True):
    if dgates is None and dlogits is None and dot is None and ids is None:
        return
    k = desc.topk
    if (dgates is not None or dlogits is not None) and (gates is None or dot is None):
        raise ValueError(f"dgates and dlogits need gates and {dot_name}")
    if dlogits is not None:
        if ids is None:
            raise ValueError("dlogits needs ids")
        _is("dlogits", dlogits, (T, desc.E), torch.float32, dev, cuda)
    if dot is not None:
        _is(dot_name, dot, dot_shape, _TORCH[desc.row_dtype], dev, cuda)
    if ids is not None:
        _is("ids", ids, (T, k), torch.int32, dev, cuda)
    if dgates is not None:
        _is("dgates", dgates, (T, k), torch.float32, dev, cuda)


def hmoe_dispatch(desc, x, perm, offsets, rows, row_slot, slot_row, row_offsets, ws, gates=None, stream=None):
    """rows[r] = (gates) x[row_slot[r] / topk], and the row maps; every output is fully written."""
    T, dev = _check_dispatch(desc, x, perm, offsets, rows, row_slot, slot_row, row_offsets, ws, gates)
    _lib.check(_lib.lib().hmoe_dispatch(ctypes.byref(desc), x.data_ptr(), T, _raw(gates), perm.data_ptr(),
                                        offsets.data_ptr(), rows.data_ptr(), row_slot.data_ptr(), slot_row.data_ptr(),
                                        row_offsets.data_ptr(), ws.data_ptr(), _bytes(ws),
                                        _raw_stream(stream, dev)))


def hmoe_dispatch_backward(desc, drows, slot_row, dx, ws, x=None, gates=None, ids=None, dgates=None, dlogits=None,
                           stream=None):
    """dx[t] = sum_j (gates) drows[slot_row[t, j]], and with gates and x the gates' and router logits' gradients."""
    T, dev = _check_collect(desc, "drows", drows, slot_row, "dx", dx, ws, gates)
    _check_gate_grads(desc, T, dev, "x", x, dx.shape, gates, ids, dgates, dlogits)
    _lib.check(_lib.lib().hmoe_dispatch_backward(ctypes.byref(desc), drows.data_ptr(), T, slot_row.data_ptr(), _raw(x),
                                                 _raw(gates), _raw(ids), dx.data_ptr(), _raw(dgates), _raw(dlogits),
                                                 ws.data_ptr(), _bytes(ws), _raw_stream(stream, dev)))


def hmoe_combine(desc, rows, slot_row, out, ws, gates=None, stream=None):
    """out[t] = sum_j (gates) rows[slot_row[t, j]]."""
    T, dev = _check_collect(desc, "rows", rows, slot_row, "out", out, ws, gates)
    _lib.check(_lib.lib().hmoe_combine(ctypes.byref(desc), rows.data_ptr(), T, slot_row.data_ptr(), _raw(gates),
                                       out.data_ptr(), ws.data_ptr(), _bytes(ws),
                                       _raw_stream(stream, dev)))


def hmoe_combine_backward(desc, dout, row_slot, slot_row, drows, ws, rows=None, gates=None, ids=None, dgates=None,
                          dlogits=None, stream=None):
    """drows[r] = (gates) dout[row_slot[r] / topk], zero on padding, and with gates and rows the gates' and router
    logits' gradients."""
    T, dev = _check_collect(desc, "drows", drows, slot_row, "dout", dout, ws, gates)
    _is("row_slot", row_slot, (drows.shape[0],), torch.int32, dev)
    _check_gate_grads(desc, T, dev, "rows", rows, drows.shape, gates, ids, dgates, dlogits)
    _lib.check(_lib.lib().hmoe_combine_backward(ctypes.byref(desc), dout.data_ptr(), T, row_slot.data_ptr(),
                                                slot_row.data_ptr(), _raw(rows), _raw(gates), _raw(ids),
                                                drows.data_ptr(), _raw(dgates), _raw(dlogits), ws.data_ptr(),
                                                _bytes(ws), _raw_stream(stream, dev)))


# ------------------------------------------------------------------ owned buffers and autograd
class RowPlan(NamedTuple):
    """The row maps of one dispatch: row_slot [R], slot_row [T, topk], row_offsets [E + 1]."""
    row_slot: torch.Tensor
    slot_row: torch.Tensor
    row_offsets: torch.Tensor


def _gate_grad_bufs(ctx, T, E, gates, gates_at, logits_at):
    dgates = torch.empty_like(gates) if ctx.needs_input_grad[gates_at] else None
    dlogits = gates.new_empty((T, E)) if ctx.needs_input_grad[logits_at] else None
    return dgates, dlogits


class _NoSecondDerivative(torch.autograd.Function):
    """The first n tensors, as if they came of the others: to differentiate them is an error."""

    @staticmethod
    def forward(ctx, n, *tensors):
        return tuple(t.detach() for t in tensors[:n])

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("the gradients of ExpertRows have no second derivative (they were used in a loss or in another "
                           "gradient, with create_graph=True)")


def _first_order(grads, given, gates, logits, dot):
    """What backward returns for its gradients (of the moved rows, the gates and the logits). Where a graph of them is
    asked for (create_graph=True), they must not pass for constants if they depend on a tensor that requires a gradient:
    the given one and the gates (through which the logits), for the gates' part also the dot products' operand."""
    if not torch.is_grad_enabled():
        return grads
    of = [given, gates, logits if gates is not None else None, dot if grads[1] is not None or grads[2] is not None else None]
    of = [t for t in of if t is not None and t.requires_grad]
    if not of:
        return grads
    live = [t for t in grads if t is not None]
    marked = iter(_NoSecondDerivative.apply(len(live), *live, *of))
    return tuple(None if t is None else next(marked) for t in grads)


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gates, logits, ids, perm, offsets, desc, ws):
        T, dev = x.shape[0], x.device
        R = hmoe_dispatch_rows(desc, T)
        rows = torch.empty((R, desc.H), dtype=x.dtype, device=dev)
        row_slot = torch.empty((R,), dtype=torch.int32, device=dev)
        slot_row = torch.empty((T, desc.topk), dtype=torch.int32, device=dev)
        row_offsets = torch.empty((desc.E + 1,), dtype=torch.int32, device=dev)
        hmoe_dispatch(desc, x, perm, offsets, rows, row_slot, slot_row, row_offsets, ws, gates=gates)
        ctx.save_for_backward(x if gates is not None else None, gates, ids, slot_row)
        ctx.desc, ctx.ws, ctx.shape, ctx.logits = desc, ws, x.shape, logits
        ctx.mark_non_differentiable(row_slot, slot_row, row_offsets)
        return rows, row_slot, slot_row, row_offsets

    @staticmethod
    def backward(ctx, drows, *_):
        x, gates, ids, slot_row = ctx.saved_tensors
        with torch.no_grad():
            d = drows.contiguous()
            dx = d.new_empty(ctx.shape)
            dgates = dlogits = None
            if gates is not None:
                dgates, dlogits = _gate_grad_bufs(ctx, ctx.shape[0], ctx.desc.E, gates, 1, 2)
            hmoe_dispatch_backward(ctx.desc, d, slot_row, dx, ctx.ws, x=x, gates=gates, ids=ids, dgates=dgates,
                                   dlogits=dlogits)
        return *_first_order((dx, dgates, dlogits), drows, gates, ctx.logits, x), None, None, None, None, None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, gates, logits, ids, row_slot, slot_row, desc, ws):
        out = rows.new_empty((slot_row.shape[0], desc.H))
        hmoe_combine(desc, rows, slot_row, out, ws, gates=gates)
        ctx.save_for_backward(rows if gates is not None else None, gates, ids, row_slot, slot_row)
        ctx.desc, ctx.ws, ctx.shape, ctx.logits = desc, ws, rows.shape, logits
        return out

    @staticmethod
    def backward(ctx, dout):
        rows, gates, ids, row_slot, slot_row = ctx.saved_tensors
        with torch.no_grad():
            d = dout.contiguous()
            drows = d.new_empty(ctx.shape)
            dgates = dlogits = None
            if gates is not None:
                dgates, dlogits = _gate_grad_bufs(ctx, d.shape[0], ctx.desc.E, gates, 1, 2)
            hmoe_combine_backward(ctx.desc, d, row_slot, slot_row, drows, ctx.ws, rows=rows, gates=gates, ids=ids,
                                  dgates=dgates, dlogits=dlogits)
        return *_first_order((drows, dgates, dlogits), dout, gates, ctx.logits, rows), None, None, None, None, None


def _check_logits(gates, ids, logits):
    """Before anything runs: logits whose gradient could not be formed, or would be left out."""
    if logits is not None and (gates is None or ids is None) and logits.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"the gradient of logits needs {'gates' if gates is None else 'ids'}")


class ExpertRows:
    """Sorting token rows by expert and bringing them back, differentiable.

    H, E, topk, dtype (bf16, fp16 or fp32), align and capacity: as in DispatchDesc.

    gates given to dispatch (or to combine) are applied there. Gradients flow to x, rows and
    gates. The gates of hmoe_plan_routes are a softmax over the chosen router logits; give ids
    and logits as well and the logits get their gradient through it (the logits' values are not
    read). Then take the gates from plan as they are: a gates tensor that requires a gradient
    itself gets one too. These are first derivatives: differentiating them again is an error.
    """

    def __init__(self, H, E, topk, max_tokens=8, dtype=torch.bfloat16, align=1, capacity=0, device="cuda"):
        if dtype not in _ROW:
            raise ValueError(f"dtype must be torch.bfloat16, torch.float16 or torch.float32, got {dtype}")
        self.desc = DispatchDesc(H, E, topk, _ROW[dtype], align, capacity)
        self.dtype = dtype
        size = hmoe_dispatch_workspace_size(self.desc, max_tokens)
        self.ws = torch.zeros(size, dtype=torch.uint8, device=device)

    def dispatch(self, x, perm, offsets, gates=None, ids=None, logits=None):
        """x [T, H] -> (rows [R, H], RowPlan)."""
        _check_logits(gates, ids, logits)
        rows, *plan = _Dispatch.apply(x, gates, logits, ids, perm, offsets, self.desc, self.ws)
        return rows, RowPlan(*plan)

    def combine(self, rows, plan, gates=None, ids=None, logits=None):
        """rows [R, H] -> out [T, H]."""
        _check_logits(gates, ids, logits)
        return _Combine.apply(rows, gates, logits, ids, plan.row_slot, plan.slot_row, self.desc, self.ws)
