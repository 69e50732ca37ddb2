"""Rotary positions of the latent grid: the angles of a token's (t, y, x), applied to queries and keys.

`rotary_plan` makes the table of a grid, `rotary` turns [B, heads, T*H*W, d] tensors by it (differentiable;
strided inputs such as a projection's token-major output come out contiguous, as `attention` takes them),
and `attention` and `attention_multi` take a plan as `rotary=`.
"""
from __future__ import annotations

import contextlib
import ctypes
from dataclasses import dataclass
from typing import Optional, Sequence, Tuple

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import _check, _dtype_code, load_library

PAIRINGS = {"adjacent": 0, "half": 1}


class SquadStrides(ctypes.Structure):
    _fields_ = [("b", ctypes.c_longlong), ("h", ctypes.c_longlong), ("n", ctypes.c_longlong)]


class SquadRotaryDesc(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int) for f in ("B", "d", "T", "H", "W", "cT", "cH", "cW", "dtype", "pairing", "inverse")]


_nothing = contextlib.nullcontext()


def on_device(dev: torch.device):
    """A context in which dev is the current device (nothing to do where it is, the common case)."""
    return _nothing if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)


def raw_stream(dev: torch.device) -> int:
    """The handle of dev's current stream."""
    return torch._C._cuda_getCurrentRawStream(dev.index)


def on_stream(stream: torch.cuda.Stream, t):
    """A context in which stream is current, for a call on t: the call allocates and launches on it."""
    if isinstance(t, torch.Tensor) and stream.device != t.device:
        raise ValueError(f"the stream is of {stream.device}, the tensors are on {t.device}")
    return torch.cuda.stream(stream)


def in_dual_level() -> bool:
    """Whether forward-mode differentiation is on: tensors may carry tangents then, without requires_grad, and only
    an autograd function (which has no formula for them, and says so) sees them."""
    return forward_ad._current_level >= 0


def has_tangent(*ts) -> bool:
    return in_dual_level() and any(t is not None and forward_ad.unpack_dual(t).tangent is not None for t in ts)


def first_order(backward):
    """once_differentiable (a second differentiation raises), without its 3 us where none can follow; a tangent of
    the incoming gradients raises too."""
    once = once_differentiable(backward)

    def run(ctx, *grads):
        if has_tangent(*grads):
            raise RuntimeError("gradients are not differentiable again: forward-mode tangents have no formula here")
        return once(ctx, *grads) if torch.is_grad_enabled() else backward(ctx, *grads)
    return run


def token_major(t: torch.Tensor) -> bool:
    """Whether a [B, heads, n, d] tensor lies in memory as [B, n, heads, d]."""
    return t.shape[1] > 1 and t.shape[2] > 1 and t.stride(1) < t.stride(2)


def empty_like_layout(t: torch.Tensor) -> torch.Tensor:
    """A dense tensor of t's shape, token-major where t is, else head-major."""
    if t.is_contiguous():
        return torch.empty_like(t)
    B, h, n, d = t.shape
    return t.new_empty_strided((B, h, n, d), (n * h * d, d, h * d, 1) if token_major(t) else (h * n * d, n * d, d, 1))


def check_strided(*named):
    """(name, tensor) pairs: CUDA tensors [B, heads, rows, d] of one dtype and device, channels contiguous."""
    ref = named[0][1]
    for name, t in named:
        if not isinstance(t, torch.Tensor) or t.dim() != 4:
            raise ValueError(f"{name} must be a [B, heads, rows, d] tensor")
        if not t.is_cuda:
            raise ValueError("libsquad needs CUDA tensors (there is no CPU path)")
        if t.dtype != ref.dtype or t.device != ref.device:
            raise ValueError(f"{name} must share {named[0][0]}'s dtype and device")
        if t.shape[3] > 1 and t.stride(3) != 1 and t.numel() > 0:
            raise ValueError(f"the channels of {name} must be contiguous (stride 1 along d)")
    _dtype_code(ref)


def as_gradient(t: torch.Tensor) -> torch.Tensor:
    """An upstream gradient as the kernels take it: as it lies where its channels are contiguous, its rows
    apart and its steps whole 16 bytes, else copied."""
    if t.is_contiguous():
        return t if t.data_ptr() % 16 == 0 else t.clone()
    d, unit = t.shape[3], 16 // t.element_size()
    fits = t.data_ptr() % 16 == 0 and (d <= 1 or t.stride(3) == 1) and all(
        size <= 1 or (step >= d and step % unit == 0) for size, step in zip(t.shape[:3], t.stride()[:3]))
    return t if fits else t.contiguous()


def default_axes(d: int) -> Tuple[int, int, int]:
    """Channels of (time, height, width): height and width a third each in whole pairs, time the rest."""
    side = 2 * (d // 6)
    return d - 2 * side, side, side


@dataclass(frozen=True, eq=False)
class Rotary:
    """The rotation of a T x H x W grid. Two plans are equal where they are one (tables are not compared).

    axes: channels turned by time, height and width (even, their sum at most d; channels past it are copied).
    table: [T*axes[0]/2 + H*axes[1]/2 + W*axes[2]/2, 2] float32 CUDA tensor of (cos, sin): per axis one row
    of pairs for each position. pairing: "adjacent" turns channels (2i, 2i+1), "half" (i, i + sum(axes)/2).
    The table is a constant: `rotary` refuses one that wants a gradient.
    """
    grid: Tuple[int, int, int]
    axes: Tuple[int, int, int]
    table: torch.Tensor
    pairing: str = "adjacent"

    def __post_init__(self):
        grid, axes, t = tuple(self.grid), tuple(self.axes), self.table
        object.__setattr__(self, "grid", grid)
        object.__setattr__(self, "axes", axes)
        if isinstance(t, torch.Tensor):  # plans are often made anew around a table: the same checks once
            key = (grid, axes, self.pairing, t.shape, t.stride(), t.dtype)
            if key in _plans:
                return
        if len(grid) != 3 or len(axes) != 3 or min(grid) < 1 or min(axes) < 0:
            raise ValueError("grid and axes are (time, height, width): positive sizes, channels of each")
        if any(c % 2 for c in axes):
            raise ValueError("axes must be even: channels turn in pairs")
        if self.pairing not in PAIRINGS:
            raise ValueError(f"pairing must be one of {sorted(PAIRINGS)}")
        rows = sum(size * (c // 2) for size, c in zip(grid, axes))
        if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or tuple(t.shape) != (rows, 2):
            raise ValueError(f"table must be float32 of shape {(rows, 2)}")
        if not t.is_contiguous():
            raise ValueError("table must be contiguous")
        if len(_plans) >= 1024:
            _plans.clear()
        _plans.add(key)


_plans = set()  # what the checks of a plan look at, of plans that passed


def rotary_plan(grid: Sequence[int], d: int, axes: Optional[Sequence[int]] = None, theta: float = 10000.0,
                offset: Sequence[float] = (0, 0, 0), pairing: str = "adjacent", device=None) -> Rotary:
    """The plan of a grid: pair i of an axis with c channels at position p turns by (offset + p) * theta^(-2i/c).

    offset: the position of the grid's first token (a later frame of a stream, a rank's first frame).
    Angles are taken in float64 on the host, so that far positions keep their accuracy.
    """
    grid = tuple(int(x) for x in grid)
    axes = default_axes(int(d)) if axes is None else tuple(int(c) for c in axes)
    if sum(axes) > d:
        raise ValueError(f"axes {axes} turn more than d={d} channels")
    if len(offset) != 3:
        raise ValueError("offset is (time, height, width)")
    parts = []
    for size, c, first in zip(grid, axes, offset):
        freq = float(theta) ** (-torch.arange(0, c, 2, dtype=torch.float64) / max(c, 1))
        ang = (torch.arange(size, dtype=torch.float64) + float(first))[:, None] * freq
        parts.append(torch.stack([ang.cos(), ang.sin()], -1).reshape(-1, 2))
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    return Rotary(grid, axes, torch.cat(parts).float().contiguous().to(dev), pairing)


_calls = {}  # kinds of the tensors and the plan -> the checked arguments of squad_rotary besides its pointers


def _rotary_call(xs, rot: Rotary, inverse: bool, ys):
    """Checks a call; returns its arguments that depend on the geometry alone."""
    c = len(xs)
    if not 1 <= c <= 2:
        raise ValueError("one or two tensors")
    check_strided(*[(f"xs[{i}]", x) for i, x in enumerate(xs)])
    ref = xs[0]
    B, _, n, d = ref.shape
    T, H, W = rot.grid
    for x in xs:
        if (x.shape[0], x.shape[2], x.shape[3]) != (B, n, d):
            raise ValueError("the tensors must share batch, tokens and d")
    if n != T * H * W:
        raise ValueError(f"n={n} but T*H*W={T * H * W}")
    if rot.table.device != ref.device:
        raise ValueError(f"the rotary table must be on {ref.device}")
    if len(ys) != c:
        raise ValueError("out must hold one tensor for each input")
    check_strided(("xs[0]", ref), *[(f"out[{i}]", y) for i, y in enumerate(ys)])
    if any(x.shape != y.shape for x, y in zip(xs, ys)):
        raise ValueError("out must hold one tensor of each input's shape")
    if any(x.numel() == 0 for x in xs):
        return None
    desc = SquadRotaryDesc(B, d, *rot.grid, *rot.axes, _dtype_code(ref), PAIRINGS[rot.pairing], int(inverse))
    return (desc, c, (ctypes.c_int * c)(*[x.shape[1] for x in xs]),
            (SquadStrides * c)(*[SquadStrides(*x.stride()[:3]) for x in xs]),
            (SquadStrides * c)(*[SquadStrides(*y.stride()[:3]) for y in ys]), ctypes.c_void_p * c)


def squad_rotary(xs: Sequence[torch.Tensor], rot: Rotary, inverse: bool = False,
                 out: Optional[Sequence[torch.Tensor]] = None, stream: Optional[torch.cuda.Stream] = None):
    """One or two tensors [B, heads, T*H*W, d] through the C ABI in one launch; returns the list of outputs.

    inverse turns by the opposite angles. out: tensors to write (any strides of whole 16-byte steps; an input
    itself for the rotation in place), else contiguous ones are made.
    """
    if not xs:
        raise ValueError("one or two tensors")
    if stream is not None:
        with on_stream(stream, xs[0]):
            return squad_rotary(xs, rot, inverse, out)
    # (empty_like is the shortest way to a contiguous tensor: 1.3 us where new_empty takes 2.4)
    ys = [torch.empty_like(x, memory_format=torch.contiguous_format) for x in xs] if out is None else list(out)
    ref, last = xs[0], xs[-1]
    # outputs made here follow from the inputs
    key = (len(xs), ref.shape, ref.stride(), ref.dtype, ref.device, last.shape, last.stride(), last.dtype, last.device,
           None if out is None else tuple([(y.shape, y.stride(), y.dtype, y.device) for y in ys]),
           rot.grid, rot.axes, rot.pairing, rot.table.device, inverse)
    try:
        call = _calls[key]
    except KeyError:
        call = _rotary_call(xs, rot, inverse, ys)
        if len(_calls) >= 1024:
            _calls.clear()
        _calls[key] = call
    if call is None:
        full = [i for i, x in enumerate(xs) if x.numel()]
        if full:  # one of the two has no heads
            squad_rotary([xs[i] for i in full], rot, inverse, [ys[i] for i in full])
        return ys
    desc, c, heads, sx, sy, pointers = call
    with on_device(ref.device):
        _check(load_library().squad_rotary(ctypes.byref(desc), c, heads, pointers(*[x.data_ptr() for x in xs]), sx,
                                           pointers(*[y.data_ptr() for y in ys]), sy, rot.table.data_ptr(),
                                           raw_stream(ref.device)), "squad_rotary")
    return ys


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rot, *xs):
        ctx.rot = rot
        ctx.save_for_backward(rot.table)
        ctx.token_major = [token_major(x) for x in xs]
        return tuple(squad_rotary(xs, rot))

    @staticmethod
    @first_order
    def backward(ctx, *grads):
        ctx.saved_tensors  # raises where the table was changed in the meantime
        take = [i for i, g in enumerate(grads) if g is not None and ctx.needs_input_grad[1 + i]]
        out = [None] * len(grads)
        if take:
            gs = [as_gradient(grads[i]) for i in take]
            ys = []
            for i, g in zip(take, gs):
                B, h, n, d = g.shape
                ys.append(g.new_empty_strided((B, h, n, d), (n * h * d, d, h * d, 1)) if ctx.token_major[i]
                          else g.new_empty(g.shape))
            for i, y in zip(take, squad_rotary(gs, ctx.rot, inverse=True, out=ys)):
                out[i] = y
        return (None, *out)


def rotary(q: torch.Tensor, k: Optional[torch.Tensor], rot: Rotary):
    """(q, k) turned by the grid's positions, as contiguous [B, heads, T*H*W, d] tensors (float32 or bfloat16).

    k may have its own number of heads, or be None (then None comes back in its place). Differentiable; the
    gradients come in the memory layout of q and k. Forward-mode tangents are refused (RuntimeError), and so is
    a table that requires a gradient or carries a tangent (ValueError; under no_grad a table may require one).
    """
    xs = (q,) if k is None else (q, k)
    if torch.is_grad_enabled() and rot.table.requires_grad or has_tangent(rot.table):
        raise ValueError("the rotary table is a constant: it has no gradient (pass table.detach())")
    # without a derivative to come there is nothing for autograd to record
    record = in_dual_level() or torch.is_grad_enabled() and any(x.requires_grad for x in xs)
    ys = _Rotary.apply(rot, *xs) if record else squad_rotary(xs, rot)
    return ys[0], None if k is None else ys[1]
