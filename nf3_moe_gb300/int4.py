"""A linear of 4-bit integer weights with a scale, and where wanted a zero point, per group (include/hmoe.h).

    linear = LinearInt4(N, K, 128, codes, scales, zeros)      # codes uint8 [N, K/2], scales and zeros [N, K/128]
    y = linear(x, bias)                                       # [T, K] -> [T, N]
"""

import ctypes

import torch
from torch.autograd.graph import increment_version

from . import _lib, _need, act_torch_dtype
from ._lib import ACT_BF16, Int4Desc
from .lora import _need_rows, _no_gradient as _no_adapter_gradient
from .rows import _INT_MAX, _forward_mode, _is, _need_constants, _raw, _raw_stream

_TORCH = {_lib.ACT_BF16: torch.bfloat16, _lib.ACT_F16: torch.float16}


def hmoe_int4_packed_size(desc):
    b = ctypes.c_size_t()
    _lib.check(_lib.lib().hmoe_int4_packed_size(ctypes.byref(desc), ctypes.byref(b)))
    return b.value


class Int4:
    """Owns the C handle of a packed 4-bit integer matrix; keeps the packed buffer alive."""

    def __init__(self, handle, desc, packed):
        self.handle, self.desc, self.packed = handle, desc, packed

    def __del__(self):
        h, self.handle = getattr(self, "handle", None), None
        if h and _lib._LIB is not None:
            _lib._LIB.hmoe_int4_destroy(h)


def _check_int4_pack(desc, codes, scales, zeros, packed, cuda=True):
    nbytes = hmoe_int4_packed_size(desc)                 # the descriptor checks (library)
    N, groups = desc.N, desc.K // desc.group
    _need("codes", codes, (N, desc.K // 2), torch.uint8, cuda=cuda)
    _need("scales", scales, (N, groups), act_torch_dtype(desc.act_dtype), device=codes.device, cuda=cuda)
    if desc.zeros:
        _need("zeros", zeros, (N, groups), torch.uint8, device=codes.device, cuda=cuda)
    elif zeros is not None:
        raise ValueError("zeros given, but the descriptor has none")
    _need("packed", packed, min_bytes=nbytes, device=codes.device, cuda=cuda)


def hmoe_int4_pack(desc, codes, scales, packed, zeros=None, stream=None):
    _check_int4_pack(desc, codes, scales, zeros, packed)
    h = ctypes.c_void_p()
    _lib.check(_lib.lib().hmoe_int4_pack(ctypes.byref(desc), codes.data_ptr(), scales.data_ptr(), _raw(zeros), packed.data_ptr(),
                                         _raw_stream(stream, codes.get_device()), ctypes.byref(h)))
    return Int4(h, desc, packed)


def _check_int4_forward(desc, x, out, bias, cuda=True):
    """Returns T, the row strides of x and out, and the device index."""
    dt, K, N = _TORCH[desc.act_dtype], desc.K, desc.N
    try:  # nearly always right: one look at all of them, and the checks below for their messages
        T, wide = x.shape
        dev = x.get_device()
        (ldx, one), (ldo, one_o) = x.stride(), out.stride()
        if T == 1:                                       # its stride is never used
            ldx, ldo = K, N
        if (wide == K and out.shape == (T, N) and x.dtype is dt is out.dtype and one == one_o == 1 and ldx >= K and ldo >= N
                and T | ldx | ldo <= _INT_MAX and (not cuda or dev >= 0 and out.get_device() == dev)
                and (bias is None or bias.shape == (N,) and bias.dtype is dt and bias.is_contiguous()
                     and (not cuda or bias.get_device() == dev))):
            return T, ldx, ldo, dev
    except (AttributeError, ValueError):
        pass
    ldx = _need_rows("x", x, None, K, dt, cuda=cuda)
    T, dev = x.shape[0], x.get_device()
    ldo = _need_rows("out", out, T, N, dt, dev, cuda)
    if bias is not None:
        _is("bias", bias, (N,), dt, dev, cuda)
    return T, ldx, ldo, dev


def _no_gradient(x, out, bias):
    _need_constants("the 4-bit integer linear has none", x=x, out=out, bias=bias)


def hmoe_int4_forward(linear, x, out, bias=None, stream=None):
    """out[t] = W x[t] (+ bias) for rows x [T, K] (a column range of a wider tensor serves) and out [T, N]. No gradient:
    x, out and bias may not require one (outside torch.no_grad())."""
    T, ldx, ldo, dev = _check_int4_forward(linear.desc, x, out, bias)
    if x.requires_grad or out.requires_grad or bias is not None and bias.requires_grad or _forward_mode():
        _no_gradient(x, out, bias)
    increment_version(out)                               # autograd does not see the library's writes
    status = _lib.lib().hmoe_int4_forward(linear.handle, x.data_ptr(), ldx, T, _raw(bias), out.data_ptr(), ldo, _raw_stream(stream, dev))
    if status:
        _lib.check(status)


class LinearInt4:
    """A linear of 4-bit integer weights with its packed matrix owned as a torch tensor.

    codes uint8 [N, K/2] (element 2i in the low nibble), scales [N, K/group] of the activation type, zeros uint8
    [N, K/group] or None (all 8): W = (q - z) s, group 32, 64 or 128. For serving: no gradient goes through it.
    max_tokens is there as in LinearW4A16; without a workspace it sizes nothing, and any batch is taken, in passes of 16
    rows that each read the weights (16 rows of 6144 x 6144 take 17 us, 4096 rows 4.2 ms).
    """

    def __init__(self, N, K, group, codes, scales, zeros=None, max_tokens=8, act_dtype=ACT_BF16, device="cuda"):
        self.desc = Int4Desc(N, K, group, 0 if zeros is None else 1, act_dtype)
        self.dtype = act_torch_dtype(act_dtype)
        self.packed = torch.empty(hmoe_int4_packed_size(self.desc), dtype=torch.uint8, device=device)
        self.linear = hmoe_int4_pack(self.desc, codes, scales, self.packed, zeros)
        self.N = N

    def __call__(self, x, bias=None, out=None, adapters=None, ids=None):
        """bias [N] of the activation type. adapters, ids: a LoraAdapters of the same widths and each row's adapter (int32
        [T], -1: none), added to the result in place."""
        if adapters is not None:
            _no_adapter_gradient(x, None, out)
        if out is None:
            out = torch.empty((x.shape[0], self.N), dtype=self.dtype, device=x.device)
        hmoe_int4_forward(self.linear, x, out, bias)
        if adapters is not None:
            adapters(x, ids, base=out, out=out)
        return out
