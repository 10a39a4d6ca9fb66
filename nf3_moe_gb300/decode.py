"""The whole layer for up to 8 tokens, from hidden states, in two kernels (include/hmoe.h).

    moe = HybridMoELayer(H, I, E, topk, bit_map, experts, max_tokens=8)
    out, ids, gates = moe.decode(x, router)          # x [T, H], router [E, H]; bias: fp32 [E] on the logits
"""

import ctypes

import torch
from torch.autograd.graph import increment_version

from . import _lib, _need
from .rows import _int32, _is, _is_ws, _need_constants, _raw, _raw_stream

DECODE_MAX_TOKENS = 8
_TORCH = {_lib.ACT_BF16: torch.bfloat16, _lib.ACT_F16: torch.float16}


def hmoe_decode_workspace_size(desc, max_tokens):
    b = ctypes.c_size_t()
    _lib.check(_lib.lib().hmoe_decode_workspace_size(ctypes.byref(desc), _int32("max_tokens", max_tokens), ctypes.byref(b)))
    return b.value


def _owned_workspace_size(desc, max_tokens):
    """Bytes of a workspace for up to max_tokens tokens (and 8), or for as many as the layer's sizes admit where that is
    less; None for a layer that hmoe_decode does not take."""
    for tokens in range(min(max_tokens, DECODE_MAX_TOKENS), -1, -1):
        try:
            return hmoe_decode_workspace_size(desc, tokens)
        except _lib.HmoeError as e:
            if _lib.STATUS_NAMES[e.status] != "HMOE_ERR_UNSUPPORTED_SHAPE":
                raise
    return None


def _check_decode(desc, x, router, out, ids, gates, ws, bias, cuda=True):
    """Returns T and the device index."""
    dt, H, E = _TORCH[desc.act_dtype], desc.H, desc.E
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"x must be a torch.Tensor, got {type(x).__name__}")
    dev = x.get_device()
    T = x.shape[0] if x.dim() == 2 else -1
    if x.shape != (T, H) or x.dtype is not dt or not x.is_contiguous() or (cuda and dev < 0):
        _need("x", x, (None, H), dt, cuda=cuda)
    _is("router", router, (E, H), dt, dev, cuda)
    _is("out", out, (T, H), dt, dev, cuda)
    if ids is not None:
        _is("ids", ids, (T, desc.topk), torch.int32, dev, cuda)
    if gates is not None:
        _is("gates", gates, (T, desc.topk), torch.float32, dev, cuda)
    if bias is not None:
        _is("bias", bias, (E,), torch.float32, dev, cuda)
    _is_ws(ws, dev, cuda)
    return T, dev


def _no_gradient(**tensors):
    """The call has no gradient: one that would lose it in silence is refused."""
    _need_constants("hmoe_decode has none", **tensors)


def hmoe_decode(layer, x, router, out, ws, bias=None, ids=None, gates=None, stream=None):
    """out [T, H] of x [T, H] through the router [E, H] (and its bias, fp32 [E]) and the experts it chooses; ids and
    gates [T, topk] are written where given. No gradient."""
    T, dev = _check_decode(layer.desc, x, router, out, ids, gates, ws, bias)
    _no_gradient(x=x, router=router, bias=bias, out=out, gates=gates)
    for t in (out, ids, gates):
        if t is not None:
            increment_version(t)                         # autograd does not see the library's writes
    status = _lib.lib().hmoe_decode(layer.handle, x.data_ptr(), T, router.data_ptr(), _raw(bias), out.data_ptr(), _raw(ids),
                                    _raw(gates), ws.data_ptr(), ws.nbytes, _raw_stream(stream, dev))
    if status:
        _lib.check(status)
