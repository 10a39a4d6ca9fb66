"""Low-rank adapters of many requests beside a shared projection (include/hmoe.h).

    adapters = LoraAdapters(K, N, slots=32, max_rank=64, max_tokens=T)
    adapters.load(3, A, B, scale=alpha / rank)       # A [rank, K], B [N, rank]
    y = linear(x)                                    # the shared projection, [T, N]
    adapters(x, ids, base=y, out=y)                  # y[t] += scale_a B_a (A_a x[t]), a = ids[t]; -1: none
"""

import ctypes

import torch
from torch.autograd.graph import increment_version

from . import _lib, _need, act_torch_dtype, hmoe_workspace_init
from ._lib import ACT_BF16, ACT_F16, LoraDesc
from .rows import _INT_MAX, _int32, _is, _is_ws, _raw_stream

_TORCH = {ACT_BF16: torch.bfloat16, ACT_F16: torch.float16}


def _need_rows(name, t, T, width, dtype, device=None, cuda=True):
    """A [T, width] tensor whose rows are contiguous and evenly spaced (a column range of a wider one serves), on the
    device of this index. Returns the row stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2 or t.shape[1] != width or (T is not None and t.shape[0] != T):
        raise ValueError(f"{name} must have shape [{'*' if T is None else T}, {width}], got {list(t.shape)}")
    if cuda and (t.get_device() < 0 or (device is not None and t.get_device() != device)):
        raise ValueError(f"{name} must be a CUDA tensor" + (f" on cuda:{device}" if device is not None else "") + f", got one on {t.device}")
    ld, one = t.stride()
    if one != 1 or (ld < width and t.shape[0] > 1):
        raise ValueError(f"the rows of {name} must be contiguous and must not overlap, got strides {list(t.stride())}")
    _int32(f"the rows of {name}", t.shape[0])
    return _int32(f"the row stride of {name}", ld) if t.shape[0] > 1 else width   # one row: its stride is never used


def _check_lora_forward(desc, x, ids, base, out, ws, cuda=True):
    """Returns T, the row strides of x, base and out, and the device index."""
    dt, K, N = _TORCH[desc.act_dtype], desc.K, desc.N
    try:  # nearly always right: one look at all of them, and the checks below for their messages
        T, wide = x.shape
        dev, row = x.get_device(), (T, N)
        (ldx, one), (ldo, one_o) = x.stride(), out.stride()
        if T == 1:                                       # its stride is never used
            ldx, ldo = K, N
        ldb, one_b = 0, 1
        if base is out:
            ldb = ldo
        elif base is not None:
            ldb, one_b = base.stride()
            if T == 1:
                ldb = N
        if (wide == K and out.shape == row and x.dtype is dt is out.dtype and one == one_o == one_b == 1
                and ldx >= K and ldo >= N and T | ldx | ldo | ldb <= _INT_MAX
                and ids.shape == (T,) and ids.dtype is torch.int32 and ids.is_contiguous() and ws.is_contiguous()
                and (not cuda or dev >= 0 and out.get_device() == ids.get_device() == ws.get_device() == dev)
                and (base is None or base is out or ldb >= N and base.dtype is dt and base.shape == row
                     and (not cuda or base.get_device() == dev))):
            return T, ldx, ldb, ldo, dev
    except (AttributeError, ValueError):
        pass
    ldx = _need_rows("x", x, None, K, dt, cuda=cuda)
    T, dev = x.shape[0], x.get_device()
    _is("ids", ids, (T,), torch.int32, dev, cuda)
    ldo = _need_rows("out", out, T, N, dt, dev, cuda)
    ldb = 0 if base is None else ldo if base is out else _need_rows("base", base, T, N, dt, dev, cuda)
    _is_ws(ws, dev, cuda)
    return T, ldx, ldb, ldo, dev


def _no_gradient(x, base, out):
    """The adapters have no gradient: a call that would lose one in silence is refused."""
    for name, t in (("x", x), ("base", base), ("out", out)):
        if getattr(t, "requires_grad", False) and torch.is_grad_enabled():
            raise RuntimeError(f"{name} requires a gradient, and the adapters have none: detach it, or call under torch.no_grad()")


def hmoe_lora_packed_size(desc):
    b = ctypes.c_size_t()
    _lib.check(_lib.lib().hmoe_lora_packed_size(ctypes.byref(desc), ctypes.byref(b)))
    return b.value


def hmoe_lora_workspace_size(desc, max_tokens):
    b = ctypes.c_size_t()
    _lib.check(_lib.lib().hmoe_lora_workspace_size(ctypes.byref(desc), _int32("max_tokens", max_tokens), ctypes.byref(b)))
    return b.value


class Lora:
    """Owns the C handle of a set of adapters; keeps the packed buffer alive."""

    def __init__(self, handle, desc, packed):
        self.handle, self.desc, self.packed = handle, desc, packed

    def __del__(self):
        h, self.handle = getattr(self, "handle", None), None
        if h and _lib._LIB is not None:
            _lib._LIB.hmoe_lora_destroy(h)


def hmoe_lora_create(desc, packed, stream=None):
    _need("packed", packed, min_bytes=hmoe_lora_packed_size(desc))
    h = ctypes.c_void_p()
    _lib.check(_lib.lib().hmoe_lora_create(ctypes.byref(desc), packed.data_ptr(), _raw_stream(stream, packed.get_device()), ctypes.byref(h)))
    return Lora(h, desc, packed)


def _check_lora_load(desc, slot, A, B, cuda=True):
    dt = act_torch_dtype(desc.act_dtype)
    _need("A", A, (None, desc.K), dt, cuda=cuda)
    _need("B", B, (desc.N, A.shape[0]), dt, device=A.device, cuda=cuda)


def hmoe_lora_load(lora, slot, A, B, scale=1.0, stream=None):
    """Put the adapter A [rank, K], B [N, rank] into a slot; A and B None empty it."""
    if A is None and B is None:
        _lib.check(_lib.lib().hmoe_lora_load(lora.handle, int(slot), None, None, 0, 0.0,
                                             _raw_stream(stream, lora.packed.get_device())))
        return
    _check_lora_load(lora.desc, slot, A, B)
    _lib.check(_lib.lib().hmoe_lora_load(lora.handle, int(slot), A.data_ptr(), B.data_ptr(), int(A.shape[0]),
                                         float(scale), _raw_stream(stream, A.get_device())))


def hmoe_lora_forward(lora, x, ids, out, ws, base=None, stream=None):
    """out[t] = base[t] + scale_a B_a (A_a x[t]), a = ids[t]; base None: zeros; base may be out. No gradient: x, base
    and out may not require one (outside torch.no_grad())."""
    T, ldx, ldb, ldo, dev = _check_lora_forward(lora.desc, x, ids, base, out, ws)
    if x.requires_grad or out.requires_grad or base is not None and base.requires_grad:
        _no_gradient(x, base, out)
    increment_version(out)                               # autograd does not see the library's writes
    status = _lib.lib().hmoe_lora_forward(lora.handle, x.data_ptr(), ldx, T, ids.data_ptr(),
                                          None if base is None else base.data_ptr(), ldb, out.data_ptr(), ldo,
                                          ws.data_ptr(), ws.nbytes, _raw_stream(stream, dev))
    if status:
        _lib.check(status)


class LoraAdapters:
    """Low-rank adapters with their packed buffer and workspace owned as torch tensors.

    K, N: widths of the projection's input and output; slots: adapters held at once; max_rank:
    the largest rank of any; max_tokens sizes the workspace. For serving, and beside trained parts as
    constants: no gradient goes through them, and a call that would need one is an error.
    """

    def __init__(self, K, N, slots, max_rank, max_tokens=8, act_dtype=ACT_BF16, device="cuda"):
        self.desc = LoraDesc(K, N, slots, max_rank, act_dtype)
        self.dtype = act_torch_dtype(act_dtype)
        self.packed = torch.empty(hmoe_lora_packed_size(self.desc), dtype=torch.uint8, device=device)
        self.lora = hmoe_lora_create(self.desc, self.packed)
        self.ws = torch.empty(hmoe_lora_workspace_size(self.desc, max_tokens), dtype=torch.uint8, device=device)
        hmoe_workspace_init(self.ws)
        self.N = N

    def load(self, slot, A, B, scale=1.0):
        hmoe_lora_load(self.lora, slot, A, B, scale)

    def unload(self, slot):
        hmoe_lora_load(self.lora, slot, None, None)

    def __call__(self, x, ids, base=None, out=None):
        if out is None:
            out = torch.empty((x.shape[0], self.N), dtype=self.dtype, device=x.device)
        hmoe_lora_forward(self.lora, x, ids, out, self.ws, base)
        return out
