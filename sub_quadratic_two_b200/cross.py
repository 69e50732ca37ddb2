"""Cross attention of the grid's tokens (or any queries) to an encoder's states of another length."""
from __future__ import annotations

import ctypes
from functools import lru_cache
from typing import Optional

import torch

from . import _check, _check_aux, _dtype_code, load_library
from .positions import (SquadStrides, as_gradient, check_strided, empty_like_layout, first_order, has_tangent,
                        in_dual_level, on_device, on_stream, raw_stream)


class SquadCrossDesc(ctypes.Structure):
    _fields_ = ([(f, ctypes.c_int) for f in ("B", "heads", "kv_heads", "n", "m", "d", "dtype")]
                + [("scale", ctypes.c_float), ("mask_stride", ctypes.c_longlong)]
                + [(f, SquadStrides) for f in ("q", "k", "v", "o", "dout", "dq", "dk", "dv")])


def _desc(q_shape, k_shape, code: int, scale: float, mask_stride: int, strides) -> SquadCrossDesc:
    B, h, n, d = q_shape
    desc = SquadCrossDesc(B, h, k_shape[1], n, k_shape[2], d, code, scale, mask_stride)
    for name, st in zip(("q", "k", "v", "o", "dout", "dq", "dk", "dv"), strides):
        setattr(desc, name, SquadStrides(*st[:3]))
    return desc


@lru_cache(maxsize=512)
def _workspace(q_shape, k_shape, code: int, which: int) -> int:
    nb = ctypes.c_size_t(0)
    desc = _desc(q_shape, k_shape, code, 0.0, 0, ())
    _check(load_library().squad_cross_workspace_size(ctypes.byref(desc), which, ctypes.byref(nb)),
           "squad_cross_workspace_size")
    return int(nb.value)


def _at(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _check_cross(q, k, v, kv_lens, key_mask) -> int:
    """Checks the operands; returns the key mask's batch stride in bytes."""
    check_strided(("q", q), ("k", k), ("v", v))
    B, h, _, d = q.shape
    if k.shape != v.shape or k.shape[0] != B or k.shape[3] != d:
        raise ValueError("k and v must be [B, kv_heads, m, d] with q's batch and d")
    if k.shape[1] == 0 or h % k.shape[1]:
        raise ValueError(f"{h} query heads are not a multiple of {k.shape[1]} key heads")
    if kv_lens is not None:
        _check_aux(kv_lens, (B,), torch.int32, q.device, "kv_lens")
    if key_mask is None:
        return 0
    m = k.shape[2]
    if not isinstance(key_mask, torch.Tensor) or key_mask.device != q.device or key_mask.dtype != torch.bool:
        raise ValueError(f"key_mask must be a bool tensor on {q.device}")
    if tuple(key_mask.shape) not in ((B, m), (1, m)) or (m > 1 and key_mask.stride(1) != 1):
        raise ValueError(f"key_mask must be [{B}, {m}] or [1, {m}] with contiguous rows")
    step = 0 if key_mask.shape[0] == 1 else key_mask.stride(0)
    if step != 0 and step < m:
        raise ValueError("the rows of key_mask must not overlap")
    return step


def _scale(scale) -> float:
    """The scale as a number (a call is kept by its value); 0 stands for 1/sqrt(d)."""
    scale = float(scale or 0.0)
    if scale < 0:
        raise ValueError("scale must be positive")
    return scale


def _kind(t: Optional[torch.Tensor]):
    """What the checks look at in a tensor."""
    return None if t is None else (t.shape, t.stride(), t.dtype, t.device)


class _Call:
    """What a checked call needs besides its pointers: the descriptor (None: nothing to launch) and the
    workspace's bytes."""
    __slots__ = ("desc", "nb")

    def __init__(self, desc, nb):
        self.desc, self.nb = desc, nb


_calls = {}  # (what the checks look at, scale) -> _Call


def _keep(key, call):
    if len(_calls) >= 1024:
        _calls.clear()
    _calls[key] = call
    return call


def _fwd_call(q, k, v, scale, kv_lens, key_mask, out) -> _Call:
    try:
        key = (q.shape, q.stride(), q.dtype, q.device, k.shape, k.stride(), k.dtype, k.device, v.shape, v.stride(),
               v.dtype, v.device, _kind(kv_lens), _kind(key_mask), _kind(out), scale)
        call = _calls.get(key)
    except (AttributeError, TypeError):  # not a tensor: the checks say which
        key = call = None
    if call is not None:
        return call
    step = _check_cross(q, k, v, kv_lens, key_mask)
    if out is not None:
        check_strided(("q", q), ("out", out))
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    o = out if out is not None else empty_like_layout(q)
    code = _dtype_code(q)
    if q.numel() == 0 or k.numel() == 0:
        call = _Call(None, 0)
    else:
        desc = _desc(q.shape, k.shape, code, scale, step, (q.stride(), k.stride(), v.stride(), o.stride()))
        call = _Call(desc, _workspace(tuple(q.shape), tuple(k.shape), code, 0))
    return _keep(key, call)


def _bwd_call(q, k, v, o, lse, dout, scale, kv_lens, key_mask) -> _Call:
    try:
        key = (q.shape, q.stride(), q.dtype, q.device, k.shape, k.stride(), k.dtype, k.device, v.shape, v.stride(),
               v.dtype, v.device, o.shape, o.stride(), o.dtype, o.device, lse.shape, lse.stride(), lse.dtype,
               lse.device, dout.shape, dout.stride(), dout.dtype, dout.device, _kind(kv_lens), _kind(key_mask), scale)
        call = _calls.get(key)
    except (AttributeError, TypeError):  # not a tensor: the checks say which
        key = call = None
    return call or _keep(key, _checked_bwd(q, k, v, o, lse, dout, scale, kv_lens, key_mask))


def _checked_bwd(q, k, v, o, lse, dout, scale, kv_lens, key_mask) -> _Call:
    step = _check_cross(q, k, v, kv_lens, key_mask)
    check_strided(("q", q), ("o", o), ("dout", dout))
    if o.shape != q.shape or dout.shape != q.shape:
        raise ValueError("o and dout must have q's shape")
    _check_aux(lse, q.shape[:3], torch.float32, q.device, "lse")
    code = _dtype_code(q)
    if q.numel() == 0 or k.numel() == 0:
        return _Call(None, 0)
    strides = [t.stride() for t in (q, k, v, o, dout)] + [empty_like_layout(t).stride() for t in (q, k, v)]
    desc = _desc(q.shape, k.shape, code, scale, step, strides)
    return _Call(desc, _workspace(tuple(q.shape), tuple(k.shape), code, 1))


def cross_workspace_size(q: torch.Tensor, k: torch.Tensor, which: int) -> int:
    """Bytes of device workspace the forward (which = 0) or backward (1) of these shapes needs."""
    return _workspace(tuple(q.shape), tuple(k.shape), _dtype_code(q), which)


def squad_cross_fwd(q, k, v, scale: Optional[float] = None, kv_lens: Optional[torch.Tensor] = None,
                    key_mask: Optional[torch.Tensor] = None, save: bool = True, out: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None):
    """Cross attention forward through the C ABI. Returns (o, lse); lse is None when save=False.

    o lies in memory as q does (token-major or head-major), or in ``out``, which must not overlap an input.
    """
    if stream is not None:
        with on_stream(stream, q):
            return squad_cross_fwd(q, k, v, scale, kv_lens, key_mask, save, out)
    scale = _scale(scale)
    return _run_fwd(_fwd_call(q, k, v, scale, kv_lens, key_mask, out), q, k, v, kv_lens, key_mask, save, out)


def _run_fwd(call, q, k, v, kv_lens, key_mask, save, out=None):
    o = empty_like_layout(q) if out is None else out
    lse = q.new_empty(q.shape[:3], dtype=torch.float32) if save else None
    if call.desc is None:  # no query, or no key for any of them
        o.zero_()
        if save:
            lse.fill_(float("-inf"))
        return o, lse
    nb = call.nb
    ws = q.new_empty(nb, dtype=torch.uint8) if nb else None
    with on_device(q.device):
        _check(load_library().squad_cross_fwd(ctypes.byref(call.desc), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                              _at(kv_lens), _at(key_mask), o.data_ptr(), _at(lse), _at(ws), nb,
                                              raw_stream(q.device)), "squad_cross_fwd")
    return o, lse


def squad_cross_bwd(q, k, v, o, lse, dout, scale: Optional[float] = None, kv_lens: Optional[torch.Tensor] = None,
                    key_mask: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """Backward through the C ABI. Returns (dq, dk, dv), each lying in memory as q, k and v do."""
    if stream is not None:
        with on_stream(stream, q):
            return squad_cross_bwd(q, k, v, o, lse, dout, scale, kv_lens, key_mask)
    call = _bwd_call(q, k, v, o, lse, dout, _scale(scale), kv_lens, key_mask)
    return _run_bwd(call, q, k, v, o, lse, dout, kv_lens, key_mask)


def _run_bwd(call, q, k, v, o, lse, dout, kv_lens, key_mask):
    dq, dk, dv = empty_like_layout(q), empty_like_layout(k), empty_like_layout(v)
    if call.desc is None:
        return dq.zero_(), dk.zero_(), dv.zero_()
    nb = call.nb
    ws = q.new_empty(nb, dtype=torch.uint8)
    with on_device(q.device):
        _check(load_library().squad_cross_bwd(ctypes.byref(call.desc), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                              _at(kv_lens), _at(key_mask), o.data_ptr(), lse.data_ptr(),
                                              dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                                              ws.data_ptr(), nb, raw_stream(q.device)), "squad_cross_bwd")
    return dq, dk, dv


class _CrossAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, scale, kv_lens, key_mask):
        o, lse = _run_fwd(_fwd_call(q, k, v, scale, kv_lens, key_mask, None), q, k, v, kv_lens, key_mask, True)
        ctx.save_for_backward(q, k, v, o, lse, kv_lens, key_mask)
        ctx.scale = scale
        return o

    @staticmethod
    @first_order
    def backward(ctx, dout):
        q, k, v, o, lse, kv_lens, key_mask = ctx.saved_tensors
        dout = as_gradient(dout)
        # hooks on saved tensors may hand them back in another layout: a call is kept for what comes back
        call = _bwd_call(q, k, v, o, lse, dout, ctx.scale, kv_lens, key_mask)
        return _run_bwd(call, q, k, v, o, lse, dout, kv_lens, key_mask) + (None, None, None)


def cross_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, scale: Optional[float] = None,
                    kv_lens: Optional[torch.Tensor] = None, key_mask: Optional[torch.Tensor] = None) -> torch.Tensor:
    """softmax(scale * q k^T) v of queries [B, heads, n, d] over states [B, kv_heads, m, d], differentiable.

    float32 or bfloat16 CUDA tensors, n and m free of each other, heads a multiple of kv_heads. Rows may be
    strided (token-major [B, n, heads, d] memory seen through transpose(1, 2)); the output lies as q does.
    scale: a positive constant, None (or 0, as in `attention`) for 1/sqrt(d); a tensor is read on the host and
    must not want a gradient (ValueError). kv_lens: [B] int32, the states of each batch row that count;
    key_mask: [B, m] (or [1, m]) bool, True where a state counts. A query with no state left gets zeros and gives
    no gradient. Gradients are not differentiable again, and forward-mode tangents are refused (RuntimeError). A
    step captured into a CUDA graph takes its gradients for leaves of its own (``t.detach().requires_grad_()``
    shares t's memory): a leaf that an eager graph still holds ties torch's autograd to the stream of that graph,
    outside the capture, and the capture fails.
    """
    if isinstance(scale, torch.Tensor) and (torch.is_grad_enabled() and scale.requires_grad or has_tangent(scale)):
        raise ValueError("scale is a constant: it has no gradient (pass float(scale))")
    if in_dual_level() or torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or v.requires_grad):
        return _CrossAttention.apply(q, k, v, _scale(scale), kv_lens, key_mask)
    return squad_cross_fwd(q, k, v, scale, kv_lens, key_mask, save=False)[0]
