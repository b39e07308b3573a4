"""Operators for sequences of tokens: embedding lookup, attention and gated
recurrence over packed frames (include/tokens.h), as a thin ctypes binding.

Tokens are pillars (``voxelize``), points (``point_map``) or the points of a
scan in spherical order (``spherical``). Frames are packed one after another;
``offsets`` is the int32 device tensor [docs + 1] of their starts and end, so a
token tensor of a fixed capacity may be passed with the offsets of what it
holds (rows outside every frame give zeros).

``embed``, ``attend`` and ``gated_scan`` are differentiable: where an input
requires a gradient they run under torch's autograd with the library's
backward kernels. ``embed_grad``, ``attend_grad`` and ``gated_scan_grad`` are
the same backward passes as plain functions, for callers that keep their own
tape or capture a step into a graph (torch's autograd must not be captured
while an eager graph of the same leaves is alive). Nothing is read back from the device and
nothing synchronised; every call works on the current stream of its tensors'
device, with outputs and workspace allocated by torch. Torch sees none of the
kernels: forward-mode derivatives and tracing raise NotImplementedError.
"""
from __future__ import annotations

import ctypes
import struct
from typing import Optional, Tuple

import torch
from torch.autograd import forward_ad
from torch.fx.experimental.proxy_tensor import get_proxy_mode

from . import VoxError, _check, library

TOK_SCAN_RUN = 16           # tokens per saved state (``carry``) of the recurrence
_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_lib = library()


class _Attention(ctypes.Structure):
    """Mirror of ``tok_attention``."""
    _fields_ = [("dtype", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("width", ctypes.c_int32),
                ("tq", ctypes.c_int64), ("tk", ctypes.c_int64),
                ("docs", ctypes.c_int32), ("mask", ctypes.c_int32),
                ("q_offsets", ctypes.c_void_p), ("k_offsets", ctypes.c_void_p),
                ("prefix", ctypes.c_void_p), ("scale", ctypes.c_float), ("cap", ctypes.c_float),
                ("slopes", ctypes.c_void_p), ("q_pos", ctypes.c_void_p),
                ("k_pos", ctypes.c_void_p), ("axes", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("q_stride", ctypes.c_int64 * 2), ("k_stride", ctypes.c_int64 * 2),
                ("v_stride", ctypes.c_int64 * 2), ("g_stride", ctypes.c_int64 * 2),
                ("q_pos_stride", ctypes.c_int64 * 2), ("k_pos_stride", ctypes.c_int64 * 2)]


# the current device's index and a device's current stream, without objects for them
_current_device, _current_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream

# The same layout, packed at once: filling the structure field by field costs
# more than the call it is for.
_PACK = struct.Struct("@4i2q2i3P2f3P2i12q")
assert _PACK.size == ctypes.sizeof(_Attention)


def _declare(lib) -> None:
    vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
    at = vp                  # tok_attention: packed bytes, or a reference to the structure
    for name, result, args in (
            ("tok_embed", i32, [vp, i64, i64, i64, i32, vp, i32, i64, f32, vp, vp]),
            ("tok_embed_grad_workspace_bytes", i64, [i64, i64, i64]),
            ("tok_embed_grad", i32, [vp, i64, i32, vp, i32, i64, i64, i64, f32, vp, vp, i64, vp]),
            ("tok_attend_workspace_bytes", i64, [at]),
            ("tok_attend_grad_workspace_bytes", i64, [at]),
            ("tok_attend", i32, [at, vp, vp, vp, vp, vp, vp, i64, vp]),
            ("tok_attend_grad", i32, [at] + [vp] * 10 + [i64, vp]),
            ("tok_scan_runs", i64, [i64]),
            ("tok_scan_workspace_bytes", i64, [i64, i64]),
            ("tok_scan", i32, [vp, vp, i32, i64, i64, vp, i32, i32] + [vp] * 5 + [i64, vp]),
            ("tok_scan_grad", i32,
             [vp, vp, vp, vp, i32, i64, i64, vp, i32, i32] + [vp] * 6 + [i64, vp])):
        f = getattr(lib, name)
        f.argtypes, f.restype = args, result


_declare(_lib)


_HALF = {torch.bfloat16: 1, torch.float16: 2}
# a proxy mode comes with a function mode, which is cheaper to ask for
_jit_tracing, _function_modes = torch._C._is_tracing, torch._C._len_torch_function_stack


def _unseen(what: str, *tensors) -> None:
    """Refuses what would lose the kernels without a word: a tangent, which the outputs would
    not carry, and tracing, which would record their allocation alone."""
    if forward_ad._current_level >= 0:
        for t in tensors:
            if isinstance(t, torch.Tensor) and forward_ad.unpack_dual(t).tangent is not None:
                raise NotImplementedError(f"{what} has no forward-mode derivative")
    if _jit_tracing() or _function_modes() and get_proxy_mode() is not None:
        raise NotImplementedError(f"{what} cannot be traced")


def _on_gpu(name: str, t: torch.Tensor, index: int = -1) -> int:
    """The index of the tensor's GPU; the one given, if one is."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    own = t.get_device()
    if own < 0:
        raise ValueError(f"{name} must be on a GPU device")
    if own != index and index >= 0:
        raise ValueError(f"{name} is on cuda:{own}, not on cuda:{index}")
    return own


def _floating(name: str, t: torch.Tensor, like: Optional[torch.Tensor] = None, types=_DTYPES) -> int:
    """The element type's code; on like's device and of its type, if it is given."""
    _on_gpu(name, t, -1 if like is None else like.get_device())
    dtype = t.dtype
    if dtype not in types:
        raise ValueError(f"{name} must be one of {', '.join(str(d) for d in types)}, not {dtype}")
    if like is not None and dtype != like.dtype:
        raise ValueError(f"{name} is {dtype}, not {like.dtype}")
    return types[dtype]


def _offsets(name: str, t: Optional[torch.Tensor], index: int) -> Optional[torch.Tensor]:
    if t is None:
        return None
    _on_gpu(name, t, index)
    if t.dtype != torch.int32 or t.dim() != 1 or t.shape[0] < 2:
        raise ValueError(f"{name} must be an int32 tensor of at least 2 offsets")
    return t.contiguous()


def _state(name: str, t: Optional[torch.Tensor], docs: int, width: int,
           index: int) -> Optional[torch.Tensor]:
    if t is None:
        return None
    _on_gpu(name, t, index)
    if t.dtype != torch.float32 or t.shape != (docs, width):
        raise ValueError(f"{name} must be a float32 tensor of shape {(docs, width)}")
    return t.contiguous()


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _address(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.data_ptr()


def _size(n: int, what: str) -> int:
    if n < 0:
        raise VoxError(int(n), what)
    return n


def _call(f, what: str, index: int, *args) -> None:
    """f(*args, stream) on the current stream of that GPU."""
    if _current_device() == index:
        rc = f(*args, _current_stream(index))
    else:
        with torch.cuda.device(index):
            rc = f(*args, _current_stream(index))
    if rc:
        _check(rc, what)


def _workspace(nbytes: int, like: torch.Tensor) -> Optional[torch.Tensor]:
    return like.new_empty(nbytes, dtype=torch.uint8) if nbytes else None


# ------------------------------------------------------------------ embedding --

def _check_ids(ids: torch.Tensor, index: int) -> torch.Tensor:
    _on_gpu("ids", ids, index)
    if ids.dtype != torch.int32 and ids.dtype != torch.int64:
        raise ValueError("ids must be int32 or int64")
    return ids.contiguous()


def _embed(table: torch.Tensor, ids: torch.Tensor, scale: float) -> torch.Tensor:
    _unseen("embed", table)
    dtype = _floating("table", table)
    index = table.get_device()
    if table.dim() != 2 or not table.numel():
        raise ValueError("table must be [rows, width]")
    ids = _check_ids(ids, index)
    rows, width = table.shape
    if table.stride(1) != 1 and width > 1 or table.stride(0) < 0:
        table = table.contiguous()
    out = table.new_empty((*ids.shape, width))
    _call(_lib.tok_embed, "tok_embed", index, table.data_ptr(), rows, width, table.stride(0), dtype,
          ids.data_ptr(), ids.element_size(), ids.numel(), scale, out.data_ptr())
    return out


def embed_grad(grad: torch.Tensor, ids: torch.Tensor, rows: int, *,
               scale: float = 1.0) -> torch.Tensor:
    """Gradient of ``embed``'s table: [rows, width] in grad's type, row r the
    sum of ``scale * grad[i]`` over the tokens i with ids[i] == r, in float32
    and in a fixed order (the same inputs give the same bits). grad is
    [*ids.shape, width]."""
    _unseen("embed_grad", grad)
    dtype = _floating("grad", grad)
    index = grad.get_device()
    ids = _check_ids(ids, index)
    if grad.shape[:-1] != ids.shape or grad.dim() < 1:
        raise ValueError(f"grad must be [*ids.shape, width]: got {tuple(grad.shape)} "
                         f"for ids {tuple(ids.shape)}")
    rows, width, n = int(rows), grad.shape[-1], ids.numel()
    flat = grad.reshape(n, width)
    if flat.stride(1) != 1 and width > 1 or flat.stride(0) < 0:
        flat = flat.contiguous()
    nbytes = _size(_lib.tok_embed_grad_workspace_bytes(n, rows, width),
                   "tok_embed_grad_workspace_bytes")
    out, ws = grad.new_empty((rows, width)), _workspace(nbytes, grad)
    _call(_lib.tok_embed_grad, "tok_embed_grad", index, flat.data_ptr(), flat.stride(0), dtype,
          ids.data_ptr(), ids.element_size(), n, rows, width, float(scale), out.data_ptr(),
          _ptr(ws), nbytes)
    return out


_GRAD_ROWS, _GRAD_TOKENS = 1 << 24, 1 << 27  # of embed_grad


class _Embed(torch.autograd.Function):
    @staticmethod
    def forward(ctx, table, ids, scale):
        if table.dim() == 2 and (table.shape[0] > _GRAD_ROWS or ids.numel() > _GRAD_TOKENS):
            raise ValueError(f"the gradient of a table holds at most {_GRAD_ROWS} rows and {_GRAD_TOKENS} "
                             f"ids: got {table.shape[0]} and {ids.numel()}")
        ctx.save_for_backward(ids)
        ctx.rows, ctx.scale = table.shape[0], scale
        return _embed(table, ids, scale)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        (ids,) = ctx.saved_tensors
        return embed_grad(grad, ids, ctx.rows, scale=ctx.scale), None, None


def embed(table: torch.Tensor, ids: torch.Tensor, *, scale: float = 1.0) -> torch.Tensor:
    """Rows of a table by token: ``scale * table[ids]``, [*ids.shape, width] in
    the table's type (float32, bf16 or fp16), rounded once. A row of zeros
    where an id is not in [0, rows) (-1 marks a point without a pillar).
    ids: int32 or int64, any shape. Differentiable in a table of at most 2^24
    rows, by at most 2^27 ids."""
    if torch.is_grad_enabled() and isinstance(table, torch.Tensor) and table.requires_grad:
        return _Embed.apply(table, ids, float(scale))
    return _embed(table, ids, float(scale))


# ------------------------------------------------------------------ attention --

def _heads(name: str, t: torch.Tensor, like: Optional[torch.Tensor] = None) -> torch.Tensor:
    _floating(name, t, like, _HALF)
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, width]")
    # 16-byte pieces, tokens less than 64 MiB apart: copy what is laid out otherwise (of no
    # tokens too, whose strides the library checks as well)
    by_token, by_head, by_element = t.stride()
    if (by_element != 1 or by_token & 7 or by_head & 7 or by_token >= 1 << 25 or t.data_ptr() & 15
            or by_token < 0 or by_head < 0):
        t = t.clone(memory_format=torch.contiguous_format)
    return t


def _positions(name: str, t: Optional[torch.Tensor], tokens: int, index: int) -> torch.Tensor:
    if t is None:
        raise ValueError(f"slopes need {name}")
    _on_gpu(name, t, index)
    if t.dtype != torch.int32 or t.dim() != 2 or t.shape[0] != tokens or not 1 <= t.shape[1] <= 3:
        raise ValueError(f"{name} must be an int32 tensor [{tokens}, 1 to 3 axes]")
    return t


def _constant(slopes) -> None:
    if isinstance(slopes, torch.Tensor) and slopes.requires_grad and torch.is_grad_enabled():
        raise ValueError("slopes are constants: no gradient is computed for them")


def _attention(q, k, v, q_offsets, k_offsets, scale, cap, slopes, q_pos, k_pos, causal, prefix,
               grad=None):
    """The checked arguments as the C structure, and the tensors it points to."""
    q, k, v = _heads("q", q), _heads("k", k, q), _heads("v", v, q)
    tq, heads, width = q.shape
    tk, kv_heads = k.shape[:2]
    if v.shape != k.shape:
        raise ValueError(f"v must have k's shape {tuple(k.shape)}, not {tuple(v.shape)}")
    if k.shape[2] != width:
        raise ValueError(f"k and v must have q's width {width}")
    if not 8 <= width <= 128 or width % 8:
        raise ValueError(f"the head width must be a multiple of 8, at most 128: got {width}")
    if heads < 1 or kv_heads < 1 or heads % kv_heads:
        raise ValueError(f"{heads} query heads cannot share {kv_heads} key heads")
    index = q.get_device()
    q_offsets, k_offsets = _offsets("q_offsets", q_offsets, index), _offsets("k_offsets", k_offsets, index)
    if (q_offsets is None) != (k_offsets is None):
        raise ValueError("pass both q_offsets and k_offsets, or neither")
    docs = 1 if q_offsets is None else q_offsets.shape[0] - 1
    if k_offsets is not None and k_offsets.shape[0] != docs + 1:
        raise ValueError("q_offsets and k_offsets must hold as many documents")
    if prefix is not None:
        _on_gpu("prefix", prefix, index)
        if prefix.dtype != torch.int32 or prefix.shape != (docs,):
            raise ValueError(f"prefix must be an int32 tensor of shape {(docs,)}")
        prefix = prefix.contiguous()
    scale = width ** -0.5 if scale is None else float(scale)
    if not 1e-30 <= scale <= 1e30:
        raise ValueError("scale must be positive: from 1e-30 to 1e30")
    if cap != 0.0 and not 2.0 ** -126 <= cap <= 2.0 ** 127:
        raise ValueError("cap must be from 2^-126 to 2^127, or 0 for none")
    axes = 0
    if slopes is not None:
        _on_gpu("slopes", slopes, index)
        if slopes.dtype != torch.float32 or slopes.shape != (heads,):
            raise ValueError(f"slopes must be a float32 tensor of shape {(heads,)}")
        slopes = slopes.contiguous()
        q_pos, k_pos = _positions("q_pos", q_pos, tq, index), _positions("k_pos", k_pos, tk, index)
        axes = q_pos.shape[1]
        if k_pos.shape[1] != axes:
            raise ValueError("q_pos and k_pos must have as many axes")
    elif q_pos is not None or k_pos is not None:
        raise ValueError("positions need slopes")
    g_stride = (0, 0)
    if grad is not None:
        grad = _heads("grad_out", grad, q)
        if grad.shape != q.shape:
            raise ValueError(f"grad_out must have q's shape {tuple(q.shape)}")
        g_stride = grad.stride()[:2]
    a = _PACK.pack(
        _DTYPES[q.dtype], heads, kv_heads, width, tq, tk, docs, bool(causal) or prefix is not None,
        _address(q_offsets), _address(k_offsets), _address(prefix), scale, cap, _address(slopes),
        _address(q_pos), _address(k_pos), axes, 0, *q.stride()[:2], *k.stride()[:2], *v.stride()[:2],
        *g_stride, *(q_pos.stride() if axes else (0, 0)), *(k_pos.stride() if axes else (0, 0)))
    return a, (q, k, v, grad, q_offsets, k_offsets, prefix, slopes, q_pos, k_pos)


def _attend(q, k, v, want_lse, **more):
    _unseen("attend", q, k, v, more["slopes"])
    a, kept = _attention(q, k, v, **more)
    q, k, v = kept[:3]
    nbytes = _size(_lib.tok_attend_workspace_bytes(a), "tok_attend_workspace_bytes")
    out, ws = q.new_empty(q.shape), _workspace(nbytes, q)
    lse = q.new_empty(q.shape[:2], dtype=torch.float32) if want_lse else None
    _call(_lib.tok_attend, "tok_attend", q.get_device(), a, q.data_ptr(), k.data_ptr(), v.data_ptr(),
          out.data_ptr(), _ptr(lse), _ptr(ws), nbytes)
    return out, lse


def attend_grad(grad_out: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                out: torch.Tensor, lse: torch.Tensor, *,
                q_offsets: Optional[torch.Tensor] = None,
                k_offsets: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                cap: float = 0.0, slopes: Optional[torch.Tensor] = None,
                q_pos: Optional[torch.Tensor] = None, k_pos: Optional[torch.Tensor] = None,
                causal: bool = False, prefix: Optional[torch.Tensor] = None
                ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Gradients of ``attend``'s q, k and v from that of its output, with the
    out and lse it returned and the same other arguments. Gradients of shared
    key heads are summed over their query heads in float32."""
    _unseen("attend_grad", grad_out, q, k, v, out, lse, slopes)
    _constant(slopes)
    a, kept = _attention(q, k, v, q_offsets, k_offsets, scale, cap, slopes, q_pos, k_pos, causal,
                         prefix, grad_out)
    q, k, v, g = kept[:4]
    _floating("out", out, q)
    _on_gpu("lse", lse, q.get_device())
    if out.shape != q.shape or lse.dtype != torch.float32 or lse.shape != q.shape[:2]:
        raise ValueError("out and lse must be what attend returned for q")
    out, lse = out.contiguous(), lse.contiguous()
    if out.data_ptr() % 16:
        out = out.clone()
    nbytes = _size(_lib.tok_attend_grad_workspace_bytes(a), "tok_attend_grad_workspace_bytes")
    gq, gk, gv = q.new_empty(q.shape), k.new_empty(k.shape), k.new_empty(k.shape)
    ws = _workspace(nbytes, q)
    _call(_lib.tok_attend_grad, "tok_attend_grad", q.get_device(), a, q.data_ptr(), k.data_ptr(), v.data_ptr(),
          out.data_ptr(), lse.data_ptr(), g.data_ptr(), gq.data_ptr(), gk.data_ptr(), gv.data_ptr(),
          _ptr(ws), nbytes)
    return gq, gk, gv


class _Attend(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, more):
        out, lse = _attend(q, k, v, True, **more)
        tensors = {n: t for n, t in more.items() if isinstance(t, torch.Tensor)}
        ctx.plain = {n: t for n, t in more.items() if n not in tensors}
        ctx.names = list(tensors)
        ctx.save_for_backward(q, k, v, out, lse, *tensors.values())
        ctx.mark_non_differentiable(lse)
        return out, lse

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad, _):
        q, k, v, out, lse, *rest = ctx.saved_tensors
        more = dict(ctx.plain, **dict(zip(ctx.names, rest)))
        return (*attend_grad(grad, q, k, v, out, lse, **more), None)


def attend(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *,
           q_offsets: Optional[torch.Tensor] = None, k_offsets: Optional[torch.Tensor] = None,
           scale: Optional[float] = None, cap: float = 0.0,
           slopes: Optional[torch.Tensor] = None, q_pos: Optional[torch.Tensor] = None,
           k_pos: Optional[torch.Tensor] = None, causal: bool = False,
           prefix: Optional[torch.Tensor] = None, return_lse: bool = False):
    """Attention inside packed documents.

    q [tq, heads, width], k and v [tk, kv_heads, width] (bf16 or fp16, heads a
    multiple of kv_heads, width a multiple of 8 up to 128), packed by
    ``q_offsets`` and ``k_offsets`` (int32 [docs + 1]; None: one document).
    Tensors are read where they are if an element's stride is 1, tokens and heads
    start at multiples of 16 bytes and tokens are less than 64 MiB apart; in any
    other layout each call copies them first.
    Scores are ``scale * q.k`` (scale None: width ** -0.5), then
    ``cap * tanh(score / cap)`` when cap > 0, then less ``slopes[head]`` times
    the L1 distance of the positions (int32 [tokens, 1 to 3 axes] in
    [0, 65535]: the coords of voxelize). ``causal`` hides the keys after a
    query (the last query sees every key); ``prefix`` (int32 [docs]) makes the
    first keys of each document visible to all its queries, and the rest causal.

    Caches with room to grow: give every cache two documents, its keys and, with
    no queries, the room left: k_offsets [0, len0, room, room + len1, 2 room, ..],
    q_offsets [0, 1, 1, 2, 2, ..]. What the room holds is not read.

    Returns out [tq, heads, width], zeros where a query sees no key, and with
    ``return_lse`` also the log-sum-exp [tq, heads] float32 (-inf there, not
    differentiable). Differentiable in q, k and v; slopes that require a gradient
    are refused unless gradients are off."""
    more = dict(q_offsets=q_offsets, k_offsets=k_offsets, scale=scale, cap=cap, slopes=slopes,
                q_pos=q_pos, k_pos=k_pos, causal=causal, prefix=prefix)
    _constant(slopes)
    if torch.is_grad_enabled() and any(isinstance(t, torch.Tensor) and t.requires_grad
                                       for t in (q, k, v)):
        out, lse = _Attend.apply(q, k, v, more)
    else:
        out, lse = _attend(q, k, v, return_lse, **more)
    return (out, lse) if return_lse else out


# ----------------------------------------------------------------- recurrence --

def _scan_args(gate, x, offsets):
    dtype = _floating("gate", gate)
    _floating("x", x, gate)
    if gate.dim() != 2 or gate.shape != x.shape or gate.shape[1] < 1:
        raise ValueError("gate and x must both be [tokens, width]")
    offsets = _offsets("offsets", offsets, gate.get_device())
    docs = 1 if offsets is None else offsets.shape[0] - 1
    return dtype, gate.contiguous(), x.contiguous(), offsets, docs


def _scan(gate, x, offsets, state, reverse, want_carry):
    _unseen("gated_scan", gate, x, state)
    dtype, gate, x, offsets, docs = _scan_args(gate, x, offsets)
    t, width = x.shape
    state = _state("state", state, docs, width, x.get_device())
    y, last = x.new_empty((t, width)), x.new_empty((docs, width), dtype=torch.float32)
    carry = None
    if want_carry:
        carry = x.new_empty((-(-t // TOK_SCAN_RUN), width), dtype=torch.float32)
    nbytes = _size(_lib.tok_scan_workspace_bytes(t, width), "tok_scan_workspace_bytes")
    ws = _workspace(nbytes, x)
    _call(_lib.tok_scan, "tok_scan", x.get_device(), gate.data_ptr(), x.data_ptr(), dtype, t, width, _ptr(offsets),
          docs, bool(reverse), _ptr(state), y.data_ptr(), last.data_ptr(), _ptr(carry), _ptr(ws), nbytes)
    return y, last, carry


def gated_scan_grad(grad_y: torch.Tensor, gate: torch.Tensor, x: torch.Tensor,
                    carry: torch.Tensor, offsets: Optional[torch.Tensor] = None, *,
                    state: Optional[torch.Tensor] = None,
                    grad_state: Optional[torch.Tensor] = None, reverse: bool = False
                    ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Gradients of ``gated_scan``'s gate, x and initial state from those of y
    and of the last state (``grad_state``, None: zeros), with the carry it
    returned and the same other arguments."""
    _unseen("gated_scan_grad", grad_y, gate, x, carry, state, grad_state)
    dtype, gate, x, offsets, docs = _scan_args(gate, x, offsets)
    t, width = x.shape
    _floating("grad_y", grad_y, x)
    if grad_y.shape != x.shape:
        raise ValueError(f"grad_y must have x's shape {tuple(x.shape)}")
    grad_y = grad_y.contiguous()
    _on_gpu("carry", carry, x.get_device())
    if carry.dtype != torch.float32 or tuple(carry.shape) != (-(-t // TOK_SCAN_RUN), width):
        raise ValueError("carry must be what gated_scan returned for x")
    carry = carry.contiguous()
    state = _state("state", state, docs, width, x.get_device())
    grad_state = _state("grad_state", grad_state, docs, width, x.get_device())
    gg, gx = gate.new_empty((t, width)), x.new_empty((t, width))
    gs = x.new_empty((docs, width), dtype=torch.float32)
    nbytes = _size(_lib.tok_scan_workspace_bytes(t, width), "tok_scan_workspace_bytes")
    ws = _workspace(nbytes, x)
    _call(_lib.tok_scan_grad, "tok_scan_grad", x.get_device(), grad_y.data_ptr(), gate.data_ptr(), x.data_ptr(),
          carry.data_ptr(), dtype, t, width, _ptr(offsets), docs, bool(reverse), _ptr(state),
          _ptr(grad_state), gg.data_ptr(), gx.data_ptr(), gs.data_ptr(), _ptr(ws), nbytes)
    return gg, gx, gs


class _GatedScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, gate, x, offsets, state, reverse):
        y, last, carry = _scan(gate, x, offsets, state, reverse, True)
        ctx.save_for_backward(gate, x, carry, offsets, state)
        ctx.reverse = reverse
        ctx.mark_non_differentiable(carry)
        return y, last, carry

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_y, grad_last, _):
        gate, x, carry, offsets, state = ctx.saved_tensors
        gg, gx, gs = gated_scan_grad(grad_y, gate, x, carry, offsets, state=state,
                                     grad_state=grad_last, reverse=ctx.reverse)
        return gg, gx, None, gs if state is not None else None, None


def gated_scan(gate: torch.Tensor, x: torch.Tensor, offsets: Optional[torch.Tensor] = None, *,
               state: Optional[torch.Tensor] = None, reverse: bool = False,
               return_carry: bool = False):
    """Gated linear recurrence along packed documents:
    ``h = a * h + (1 - a) * x`` with ``a = sigmoid(gate)``, per channel.

    gate and x [tokens, width] (float32, bf16 or fp16), packed by ``offsets``
    (int32 [docs + 1]; None: one document); ``state`` [docs, width] float32 is
    h before each document's first token (None: zeros). ``reverse`` runs from
    each document's last token to its first.

    Returns (y [tokens, width] in x's type: h at every token; the states after
    each document's last step [docs, width] float32), and with
    ``return_carry`` the saved states that ``gated_scan_grad`` takes. One call
    with documents of one token each is a step of decoding. Differentiable in
    gate, x and state."""
    if torch.is_grad_enabled() and any(isinstance(t, torch.Tensor) and t.requires_grad
                                       for t in (gate, x, state)):
        y, last, carry = _GatedScan.apply(gate, x, offsets, state, bool(reverse))
    else:
        y, last, carry = _scan(gate, x, offsets, state, reverse, return_carry)
    return (y, last, carry) if return_carry else (y, last)
