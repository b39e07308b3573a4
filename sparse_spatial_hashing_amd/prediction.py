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
from typing import Optional, Tuple

import torch

from .tokens import (_HALF, _call, _check_ids, _floating, _lib, _on_gpu, _ptr, _size, _unseen,
                     _workspace)


def _declare(lib) -> None:
    vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
    loss = [vp, i64, vp, i64, i32, i64, i64, i64, vp, i32]
    for name, result, args in (
            ("tok_rotate", i32, [vp] + [i64] * 5 + [i32, vp, i64, i64, i32, vp, i64, i32, i32, vp, vp]),
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
    _unseen("rotate", x)
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
    shape and type, rounded once. Differentiable in x."""
    if torch.is_grad_enabled() and isinstance(x, torch.Tensor) and x.requires_grad:
        return _Rotate.apply(x, pos, freqs, bool(interleaved), bool(inverse))
    return _rotate(x, pos, freqs, bool(interleaved), bool(inverse))


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
    gx, gt = x.new_empty((t, width)), x.new_empty((rows, width))
    ws = _workspace(nbytes, x)
    _call(_lib.tok_row_loss_grad, "tok_row_loss_grad", index, grad_loss.data_ptr(), *args, lse.data_ptr(), scale,
          gx.data_ptr(), gt.data_ptr(), _ptr(ws), nbytes)
    if width != x.shape[-1]:
        gx, gt = gx[:, :x.shape[-1]].contiguous(), gt[:, :x.shape[-1]].contiguous()
    return gx.view(x.shape), gt


class _RowLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, table, ids, scale):
        loss, lse = _row_loss(x, table, ids, scale, True)
        ctx.save_for_backward(x, table, ids, lse)
        ctx.scale = scale
        ctx.mark_non_differentiable(lse)
        return loss, lse

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad, _):
        gx, gt = row_loss_grad(grad, *ctx.saved_tensors, scale=ctx.scale)
        return gx, gt, None, None


def row_loss(x: torch.Tensor, table: torch.Tensor, ids: torch.Tensor, *, scale: float = 1.0,
             return_lse: bool = False):
    """The loss of predicting rows of a table, token by token: the log of the sum
    over all rows of ``exp(scale * x.row)``, less ``scale * x.table[id]``.

    x [*ids.shape, width] and table [rows, width] (bf16 or fp16: the table of
    ``embed``, or a product's weight), ids int32 or int64. float32 [*ids.shape]; 0
    where an id is not in [0, rows), and nothing passes to or from that token.
    Logits are never in memory as a whole: their workspace grows with the tokens
    and stays under some hundred MiB. With ``return_lse`` also the log of the sum
    (float32, 0 without a row, not differentiable). A width that is no multiple of 8
    is copied into one that is, by each call; so are rows off 16 bytes or 8 MiB and
    more apart. Differentiable in x and table, always both."""
    if torch.is_grad_enabled() and any(isinstance(v, torch.Tensor) and v.requires_grad for v in (x, table)):
        loss, lse = _RowLoss.apply(x, table, ids, scale)
    else:
        loss, lse = _row_loss(x, table, ids, scale, return_lse)
    return (loss, lse) if return_lse else loss
