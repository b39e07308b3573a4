"""Operators of a model that predicts tokens, next to those of ``tokens``: rotary
positions, attention with decay, and the loss over the rows of a table
(include/tokens.h), as a thin ctypes binding with the same conventions.

``rotate`` turns queries and keys by their places (on the grid, or along the
frame) before ``attend``; ``decay_attend`` mixes tokens at a cost that grows with
their number alone, and one token at a time when a model is asked; ``row_loss``
compares what comes out with every row of ``embed``'s table.

All are differentiable under torch's autograd; ``decay_attend_grad`` and
``row_loss_grad`` are the backward passes as plain functions (``rotate``'s is
``rotate`` with ``inverse``).
"""
from __future__ import annotations

import ctypes
import math
import struct
from typing import Optional, Tuple

import torch

from .tokens import (_DTYPES, _HALF, _address, _call, _check_ids, _floating, _heads, _lib,
                     _offsets, _on_gpu, _ptr, _size, _unseen, _workspace)


class _Decay(ctypes.Structure):
    """Mirror of ``tok_decay``."""
    _fields_ = [("dtype", ctypes.c_int32), ("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("width", ctypes.c_int32), ("t", ctypes.c_int64), ("docs", ctypes.c_int32),
                ("reverse", ctypes.c_int32), ("offsets", ctypes.c_void_p), ("decay", ctypes.c_void_p),
                ("scale", ctypes.c_float), ("reserved", ctypes.c_int32),
                ("q_stride", ctypes.c_int64 * 2), ("k_stride", ctypes.c_int64 * 2),
                ("v_stride", ctypes.c_int64 * 2), ("g_stride", ctypes.c_int64 * 2)]


# the same layout, packed at once
_PACK = struct.Struct("@4iq2i2Pfi8q")
assert _PACK.size == ctypes.sizeof(_Decay)


def _declare(lib) -> None:
    vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
    loss = [vp, i64, vp, i64, i32, i64, i64, i64, vp, i32]
    for name, result, args in (
            ("tok_rotate", i32, [vp] + [i64] * 5 + [i32, vp, i64, i64, i32, vp, i64, i32, i32, vp, vp]),
            ("tok_decay_carry_rows", i64, [vp]),
            ("tok_decay_grad_workspace_bytes", i64, [vp]),
            ("tok_decay_attend", i32, [vp] * 9),
            ("tok_decay_attend_grad", i32, [vp] * 13 + [i64, vp]),
            ("tok_row_loss_workspace_bytes", i64, [i64] * 3),
            ("tok_row_loss_grad_workspace_bytes", i64, [i64] * 3),
            ("tok_row_loss", i32, loss + [f32, vp, vp, vp, i64, vp]),
            ("tok_row_loss_grad", i32, [vp] + loss + [vp, f32, vp, vp, vp, i64, vp])):
        f = getattr(lib, name)
        f.argtypes, f.restype = args, result


_declare(_lib)


# ------------------------------------------------------------ rotary positions --

def rotary_frequencies(rotated: int, *, base: float = 10000.0, axes: int = 1, stretch: float = 1.0,
                       context: float = 0.0, turns: Tuple[float, float] = (1.0, 32.0),
                       device="cuda") -> torch.Tensor:
    """Radians per position for ``rotate``: float64 [axes, rotated / (2 axes)], the
    same for every axis, ``base ** (-pair / pairs)``.

    ``stretch`` > 1 scales them for contexts that much longer than the model was
    trained with: all by 1 / stretch (positions squeezed), or with ``context``
    (positions it was trained with) by how often a pair turns within them: up to
    turns[0] times by 1 / stretch, from turns[1] times on not at all, between the
    two by what lies between."""
    rotated, axes = int(rotated), int(axes)
    if not 1 <= axes <= 3 or rotated < 2 * axes or rotated % (2 * axes):
        raise ValueError(f"{rotated} elements are no pairs for each of {axes} axes (1 to 3)")
    low, high = (float(v) for v in turns)
    if not (base > 0 and stretch >= 1 and context >= 0 and high > low >= 0) or \
            not all(map(math.isfinite, (base, stretch, context, high))):
        raise ValueError("base must be positive, stretch at least 1, context not negative, turns increasing")
    pairs = rotated // (2 * axes)
    f = [float(base) ** (-p / pairs) for p in range(pairs)]
    if stretch != 1:
        for p, x in enumerate(f):
            kept = (context * x / (2 * math.pi) - low) / (high - low) if context else 0.0
            kept = min(1.0, max(0.0, kept))
            f[p] = x * ((1.0 - kept) / stretch + kept)
    return torch.tensor([f] * axes, dtype=torch.float64, device=device)


def _rotate(x, pos, freqs, interleaved, inverse):
    _unseen("rotate", x, freqs)
    dtype = _floating("x", x)
    index = x.get_device()
    if x.dim() != 3 or x.shape[1] < 1 or x.shape[2] < 1:
        raise ValueError("x must be [tokens, heads, width]")
    _on_gpu("pos", pos, index)
    tokens, heads, width = x.shape
    if pos.dtype != torch.int32 or pos.dim() not in (1, 2) or pos.shape[0] != tokens:
        raise ValueError(f"pos must be an int32 tensor [{tokens}] or [{tokens}, axes]")
    axes = pos.shape[1] if pos.dim() == 2 else 1
    _on_gpu("freqs", freqs, index)
    if freqs.dtype != torch.float64 or freqs.dim() != 2 or freqs.shape[0] != axes or not 1 <= axes <= 3:
        raise ValueError(f"freqs must be a float64 tensor [axes, pairs] for the {axes} axes of pos (1 to 3)")
    pairs = freqs.shape[1]
    if pairs < 1 or 2 * axes * pairs > width:
        raise ValueError(f"{axes} axes of {pairs} pairs do not fit a width of {width}")
    freqs = freqs.contiguous()
    by_token, by_head, by_element = x.stride()
    if by_element != 1 or by_token < 0 or by_head < 0:
        x = x.contiguous()
        by_token, by_head = x.stride()[:2]
    out = x.new_empty((tokens, heads, width))
    _call(_lib.tok_rotate, "tok_rotate", index, x.data_ptr(), tokens, heads, width, by_token, by_head, dtype,
          pos.data_ptr(), pos.stride(0), pos.stride(1) if pos.dim() == 2 else 1, axes, freqs.data_ptr(), pairs,
          interleaved, inverse, out.data_ptr())
    return out


class _Rotate(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, pos, freqs, interleaved, inverse):
        ctx.save_for_backward(pos, freqs)
        ctx.how = interleaved, inverse
        return _rotate(x, pos, freqs, interleaved, inverse)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        pos, freqs = ctx.saved_tensors
        interleaved, inverse = ctx.how
        return _rotate(grad, pos, freqs, interleaved, not inverse), None, None, None, None


def rotate(x: torch.Tensor, pos: torch.Tensor, freqs: torch.Tensor, *, interleaved: bool = False,
           inverse: bool = False) -> torch.Tensor:
    """Rotary positions: pairs of a head's elements turned by position * frequency.

    x [tokens, heads, width] (float32, bf16 or fp16; queries and keys of one
    product may go through one call as a view of it), pos int32 [tokens] or
    [tokens, 1 to 3 axes] (any values: the coords of voxelize, or the places along
    a frame), freqs float64 [axes, pairs] (``rotary_frequencies``). Axis c turns
    the 2 * pairs elements of every head from 2 * c * pairs on, element p with
    element pairs + p, or ``interleaved`` 2 p with 2 p + 1; the rest of the head is
    copied. ``inverse`` turns the other way. Returns a contiguous tensor of x's
    shape and type, rounded once. Differentiable in x; freqs that require a gradient are
    refused unless gradients are off."""
    if isinstance(freqs, torch.Tensor) and freqs.requires_grad and torch.is_grad_enabled():
        raise ValueError("freqs are constants: no gradient is computed for them")
    if torch.is_grad_enabled() and isinstance(x, torch.Tensor) and x.requires_grad:
        return _Rotate.apply(x, pos, freqs, bool(interleaved), bool(inverse))
    return _rotate(x, pos, freqs, bool(interleaved), bool(inverse))


# -------------------------------------------------------- attention with decay --

def _states(name: str, t: Optional[torch.Tensor], shape, index: int) -> Optional[torch.Tensor]:
    if t is None:
        return None
    _on_gpu(name, t, index)
    if t.dtype != torch.float32 or t.shape != shape:
        raise ValueError(f"{name} must be a float32 tensor of shape {shape}")
    t = t.contiguous()
    return t.clone() if t.data_ptr() & 15 else t


def _decay_args(q, k, v, decay, offsets, scale, reverse, grad=None):
    """The checked arguments as the C structure, the tensors it points to, the documents, and
    the states' shape."""
    q, k, v = _heads("q", q), _heads("k", k, q), _heads("v", v, q)
    t, heads, width = q.shape
    kv_heads = k.shape[1]
    if v.shape != k.shape or k.shape[0] != t or k.shape[2] != width:
        raise ValueError(f"k and v must be [tokens, heads, width] for q's tokens and width: got {tuple(k.shape)} "
                         f"and {tuple(v.shape)} for {tuple(q.shape)}")
    if not 8 <= width <= 128 or width % 8:
        raise ValueError(f"the head width must be a multiple of 8, at most 128: got {width}")
    if heads < 1 or kv_heads < 1 or heads % kv_heads:
        raise ValueError(f"{heads} query heads cannot share {kv_heads} key heads")
    index = q.get_device()
    _on_gpu("decay", decay, index)
    if decay.dtype != torch.float32 or decay.shape != (heads,):
        raise ValueError(f"decay must be a float32 tensor of shape {(heads,)}")
    decay, offsets = decay.contiguous(), _offsets("offsets", offsets, index)
    docs = 1 if offsets is None else offsets.shape[0] - 1
    scale = width ** -0.5 if scale is None else float(scale)
    if not 1e-30 <= scale <= 1e30:
        raise ValueError("scale must be positive: from 1e-30 to 1e30")
    g_stride = (0, 0)
    if grad is not None:
        grad = _heads("grad_out", grad, q)
        if grad.shape != q.shape:
            raise ValueError(f"grad_out must have q's shape {tuple(q.shape)}")
        g_stride = grad.stride()[:2]
    a = _PACK.pack(_DTYPES[q.dtype], heads, kv_heads, width, t, docs, bool(reverse), _address(offsets),
                   decay.data_ptr(), scale, 0, *q.stride()[:2], *k.stride()[:2], *v.stride()[:2], *g_stride)
    return a, (q, k, v, grad, decay, offsets), (docs, heads, width, width)


def _decay_attend(q, k, v, decay, offsets, state, scale, reverse, want_state):
    _unseen("decay_attend", q, k, v, decay, state)
    a, kept, shape = _decay_args(q, k, v, decay, offsets, scale, reverse)
    q, k, v = kept[:3]
    state = _states("state", state, shape, q.get_device())
    rows = _size(_lib.tok_decay_carry_rows(a), "tok_decay_carry_rows")
    out = q.new_empty(q.shape)
    last = q.new_empty(shape, dtype=torch.float32) if want_state else None
    carry = q.new_empty((rows, *shape[1:]), dtype=torch.float32)
    _call(_lib.tok_decay_attend, "tok_decay_attend", q.get_device(), a, q.data_ptr(), k.data_ptr(), v.data_ptr(),
          _ptr(state), out.data_ptr(), _ptr(last), carry.data_ptr())
    return out, last, carry


def decay_attend_grad(grad_out: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                      decay: torch.Tensor, carry: torch.Tensor, offsets: Optional[torch.Tensor] = None, *,
                      state: Optional[torch.Tensor] = None, grad_state: Optional[torch.Tensor] = None,
                      scale: Optional[float] = None, reverse: bool = False):
    """Gradients of ``decay_attend``'s q, k, v and initial state (None without one) from
    those of its output and of the last state (``grad_state``, None: zeros), with the carry
    it returned and the same other arguments. Gradients of shared key heads are summed over
    their query heads in float32, for which a call takes 8 bytes an element of q."""
    _unseen("decay_attend_grad", grad_out, q, k, v, decay, carry, state, grad_state)
    a, kept, shape = _decay_args(q, k, v, decay, offsets, scale, reverse, grad_out)
    q, k, v, g = kept[:4]
    index = q.get_device()
    state, grad_state = _states("state", state, shape, index), _states("grad_state", grad_state, shape, index)
    rows = _size(_lib.tok_decay_carry_rows(a), "tok_decay_carry_rows")
    carry = _states("carry", carry, (rows, *shape[1:]), index)
    if carry is None:
        raise ValueError("carry must be what decay_attend returned")
    nbytes = _size(_lib.tok_decay_grad_workspace_bytes(a), "tok_decay_grad_workspace_bytes")
    gq, gk, gv = q.new_empty(q.shape), k.new_empty(k.shape), v.new_empty(v.shape)
    gs = None if state is None else torch.empty_like(state)
    ws = _workspace(nbytes, q)
    _call(_lib.tok_decay_attend_grad, "tok_decay_attend_grad", index, a, q.data_ptr(), k.data_ptr(), v.data_ptr(),
          g.data_ptr(), _ptr(state), carry.data_ptr(), _ptr(grad_state), gq.data_ptr(), gk.data_ptr(), gv.data_ptr(),
          _ptr(gs), _ptr(ws), nbytes)
    return gq, gk, gv, gs


class _DecayAttend(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, decay, offsets, state, scale, reverse, want_state):
        out, last, carry = _decay_attend(q, k, v, decay, offsets, state, scale, reverse, want_state)
        ctx.save_for_backward(q, k, v, decay, carry, offsets, state)
        ctx.how = dict(scale=scale, reverse=reverse)
        ctx.mark_non_differentiable(carry)
        ctx.set_materialize_grads(False)  # no zeros for a state that nothing used, nor for carry
        return out, last, carry

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad, grad_last, _):
        if grad is None and grad_last is None:
            return (None,) * 9
        q, k, v, decay, carry, offsets, state = ctx.saved_tensors
        if grad is None:
            grad = q.new_zeros(q.shape)
        gq, gk, gv, gs = decay_attend_grad(grad, q, k, v, decay, carry, offsets, state=state, grad_state=grad_last,
                                           **ctx.how)
        return gq, gk, gv, None, None, gs, None, None, None


def decay_attend(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, decay: torch.Tensor,
                 offsets: Optional[torch.Tensor] = None, *, state: Optional[torch.Tensor] = None,
                 scale: Optional[float] = None, reverse: bool = False, return_state: bool = True,
                 return_carry: bool = False):
    """Attention whose weights fall with the distance along a document alone, at a cost
    that grows with the tokens: ``S = exp(-decay) S + k v^T; out = scale * q S`` per head.

    q [tokens, heads, width], k and v [tokens, kv_heads, width] (bf16 or fp16, heads a
    multiple of kv_heads, width a multiple of 8 up to 128; layouts as for ``attend``),
    packed by ``offsets`` (int32 [docs + 1]; None: one document). decay float32 [heads],
    not negative (0 forgets nothing); scale None: width ** -0.5. ``state`` float32
    [docs, heads, width, width] (of k's elements by v's) is S before each document's first
    token (None: zeros). ``reverse`` runs from each document's last token to its first.

    Returns (out [tokens, heads, width], zeros outside every document; the states after each
    document's last step, or None without ``return_state``), and with ``return_carry`` the
    saved states that ``decay_attend_grad`` takes. One call with documents of one token
    each is a step of decoding. Differentiable in q, k, v and state; a decay that requires
    a gradient is refused unless gradients are off."""
    if isinstance(decay, torch.Tensor) and decay.requires_grad and torch.is_grad_enabled():
        raise ValueError("decay is a constant: no gradient is computed for it")
    if torch.is_grad_enabled() and any(isinstance(t, torch.Tensor) and t.requires_grad for t in (q, k, v, state)):
        out, last, carry = _DecayAttend.apply(q, k, v, decay, offsets, state, scale, bool(reverse), bool(return_state))
    else:
        out, last, carry = _decay_attend(q, k, v, decay, offsets, state, scale, bool(reverse), return_state)
    return (out, last, carry) if return_carry else (out, last)


# ------------------------------------------------------------------------ loss --

def _rows(name: str, t: torch.Tensor, width: int) -> torch.Tensor:
    """As the kernels read it: rows of 16-byte pieces, less than 8 MiB apart."""
    if width % 8:
        return torch.nn.functional.pad(t, (0, 8 - width % 8))
    by_row, by_element = t.stride()
    if by_element != 1 or by_row & 7 or not 0 <= by_row < 1 << 22 or t.data_ptr() & 15:
        t = t.clone(memory_format=torch.contiguous_format)
    return t


def _loss_args(x, table, ids, scale):
    dtype = _floating("x", x, None, _HALF)
    _floating("table", table, x, _HALF)
    index = x.get_device()
    ids = _check_ids(ids, index)
    if table.dim() != 2 or not table.numel():
        raise ValueError("table must be [rows, width]")
    rows, width = table.shape
    if x.dim() < 1 or tuple(x.shape) != (*ids.shape, width):
        raise ValueError(f"x must be [*ids.shape, width]: got {tuple(x.shape)} for ids {tuple(ids.shape)} "
                         f"and a table of width {width}")
    scale = float(scale)
    if not 1e-30 <= scale <= 1e30:
        raise ValueError("scale must be positive: from 1e-30 to 1e30")
    t = ids.numel()
    x, table = _rows("x", x.reshape(t, width), width), _rows("table", table, width)
    width = table.shape[1]
    return (x, table, ids), (x.data_ptr(), x.stride(0), table.data_ptr(), table.stride(0), dtype, t, rows, width,
                             ids.data_ptr(), ids.element_size()), scale


def _row_loss(x, table, ids, scale, want_lse):
    _unseen("row_loss", x, table)
    kept, args, scale = _loss_args(x, table, ids, scale)
    t, rows, width = args[5:8]
    nbytes = _size(_lib.tok_row_loss_workspace_bytes(t, rows, width), "tok_row_loss_workspace_bytes")
    loss = x.new_empty(ids.shape, dtype=torch.float32)
    lse = torch.empty_like(loss) if want_lse else None
    ws = _workspace(nbytes, x)
    _call(_lib.tok_row_loss, "tok_row_loss", x.get_device(), *args, scale, loss.data_ptr(), _ptr(lse), _ptr(ws),
          nbytes)
    return loss, lse


def row_loss_grad(grad_loss: torch.Tensor, x: torch.Tensor, table: torch.Tensor, ids: torch.Tensor,
                  lse: torch.Tensor, *, scale: float = 1.0) -> Tuple[torch.Tensor, torch.Tensor]:
    """Gradients of ``row_loss``'s x and table from that of the loss (float32
    [*ids.shape]), with the lse it returned and the same other arguments."""
    return _row_loss_grad(grad_loss, x, table, ids, lse, scale, True, True)


def _row_loss_grad(grad_loss, x, table, ids, lse, scale, want_x, want_table):
    _unseen("row_loss_grad", grad_loss, x, table, lse)
    kept, args, scale = _loss_args(x, table, ids, scale)
    t, rows, width = args[5:8]
    index = x.get_device()
    for name, v in (("grad_loss", grad_loss), ("lse", lse)):
        _on_gpu(name, v, index)
        if v.dtype != torch.float32 or v.shape != ids.shape:
            raise ValueError(f"{name} must be a float32 tensor of shape {tuple(ids.shape)}")
    grad_loss, lse = grad_loss.contiguous(), lse.contiguous()
    nbytes = _size(_lib.tok_row_loss_grad_workspace_bytes(t, rows, width), "tok_row_loss_grad_workspace_bytes")
    gx = x.new_empty((t, width)) if want_x else None
    gt = x.new_empty((rows, width)) if want_table else None
    ws = _workspace(nbytes, x)
    _call(_lib.tok_row_loss_grad, "tok_row_loss_grad", index, grad_loss.data_ptr(), *args, lse.data_ptr(), scale,
          _address(gx), _address(gt), _ptr(ws), nbytes)
    gx, gt = (g if g is None or width == x.shape[-1] else g[:, :x.shape[-1]].contiguous() for g in (gx, gt))
    return None if gx is None else gx.view(x.shape), gt


class _RowLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, table, ids, scale):
        loss, lse = _row_loss(x, table, ids, scale, True)
        ctx.save_for_backward(x, table, ids, lse)
        ctx.scale = scale
        ctx.mark_non_differentiable(lse)
        ctx.set_materialize_grads(False)  # no zeros for lse
        return loss, lse

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad, _):
        if grad is None:
            return (None,) * 4
        gx, gt = _row_loss_grad(grad, *ctx.saved_tensors, ctx.scale, *ctx.needs_input_grad[:2])
        return gx, gt, None, None


def row_loss(x: torch.Tensor, table: torch.Tensor, ids: torch.Tensor, *, scale: float = 1.0,
             return_lse: bool = False):
    """The loss of predicting rows of a table, token by token: the log of the sum
    over all rows of ``exp(scale * x.row)``, less ``scale * x.table[id]``.

    x [*ids.shape, width] and table [rows, width] (bf16 or fp16: the table of
    ``embed``, or a product's weight), ids int32 or int64. float32 [*ids.shape]; 0
    where an id is not in [0, rows), and nothing passes to or from that token.
    Logits are never in memory as a whole: a call's workspace is x once more where it is
    wider than 128 (to whole 256s), the gradients' that and x in float32 (six bytes an
    element and a little more), 12 bytes a token, and up to 768 MiB besides (three times as
    much at widths over 4096). With ``return_lse`` also the log of the sum
    (float32, 0 without a row, not differentiable). A width that is no multiple of 8
    is copied into one that is, by each call; so are rows off 16 bytes or 8 MiB and
    more apart. Differentiable in x and table; what needs no gradient costs none."""
    if torch.is_grad_enabled() and any(isinstance(v, torch.Tensor) and v.requires_grad for v in (x, table)):
        loss, lse = _RowLoss.apply(x, table, ids, scale)
    else:
        loss, lse = _row_loss(x, table, ids, scale, return_lse)
    return (loss, lse) if return_lse else loss
