"""The operators of models that predict tokens from their definitions, in 64 bits
on the CPU, with a bound on what a kernel that follows include/tokens.h may differ
by (as token_reference: `u` is half a step of the tensors' type, E that of float32)."""
import math

import torch

from token_reference import E, unit


# ------------------------------------------------------------ rotary positions --

def rotate(x, pos, freqs, interleaved=False, inverse=False):
    pos = pos[:, None] if pos.dim() == 1 else pos
    axes, pairs = freqs.shape
    z, out, size = x.double(), x.double().clone(), torch.zeros(x.shape, dtype=torch.float64)
    for c in range(axes):
        p = torch.arange(pairs)
        first = 2 * pairs * c + (2 * p if interleaved else p)
        second = first + (1 if interleaved else pairs)
        angle = pos[:, c, None].double() * freqs[c].double() * (-1 if inverse else 1)
        cos, sin = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
        u, v = z[:, :, first], z[:, :, second]
        out[:, :, first], out[:, :, second] = u * cos - v * sin, u * sin + v * cos
        size[:, :, first] = size[:, :, second] = u.abs() + v.abs()
    # the turn in float32 (2^-26 of 2 pi), its sine and cosine (2 steps), two products and a sum;
    # in 64 bits a turn is right to 2^-52 of its size
    far = float((pos.double().abs()[:, :, None] * freqs).max()) if pos.numel() else 0.0
    bound = size * (16 * E + far * 2.0 ** -51) + out.abs() * unit(x.dtype)
    return out, torch.where(size > 0, bound + torch.finfo(x.dtype).smallest_normal, 0.0)


# ------------------------------------------------------------------------ loss --

def row_loss(x, table, ids, scale, grad=None):
    """{"loss", "lse" and with grad "gx", "gt"}: (value, bound). x [t, width], ids [t]."""
    u = unit(x.dtype)
    rows, width = table.shape
    ids = ids.long()
    has = (ids >= 0) & (ids < rows)
    y, w = x[has].double(), table.double()
    came = ids[has]
    z = scale * y @ w.T
    # a product of `width` terms in any order; its scaling, the difference in the exponent
    off = E * (width + 8) * scale * (y.abs() @ w.abs().T) + 8 * E * (z.abs() + 1)
    lse = torch.logsumexp(z, 1)
    p = torch.exp(z - lse[:, None])
    # a weight's relative error: its score's and the largest's, the sum's of `rows` terms
    off = off + 4 * E * lse.abs()[:, None]
    lse_off = (p * off).sum(1) + E * (rows + 16)
    hit = z.gather(1, came[:, None])[:, 0]
    hit_off = off.gather(1, came[:, None])[:, 0]
    t = x.shape[0]
    val = {"loss": torch.zeros(t, dtype=torch.float64), "lse": torch.zeros(t, dtype=torch.float64)}
    tol = {n: torch.zeros(t, dtype=torch.float64) for n in val}
    val["lse"][has], tol["lse"][has] = lse, lse_off + 4 * E * lse.abs()
    val["loss"][has] = lse - hit
    tol["loss"][has] = lse_off + hit_off + 4 * E * (lse.abs() + hit.abs())
    if grad is not None:
        g = grad.double()[has]
        one = torch.zeros_like(p)
        one[torch.arange(len(came)), came] = 1.0
        b = (p - one) * g[:, None]
        r = off + lse_off[:, None] + 16 * E
        b_off = p * g.abs()[:, None] * r + b.abs() * (u + 4 * E)
        if x.dtype == torch.float16 and g.numel():
            b_off = b_off + 2.0 ** -37 * g.abs().max()  # half the smallest step, lifted by 2^13 at least
        small = torch.finfo(x.dtype).smallest_normal
        val["gx"], tol["gx"] = (torch.zeros(x.shape, dtype=torch.float64) for _ in range(2))
        val["gx"][has] = scale * b @ w
        tol["gx"][has] = scale * ((b_off + E * (rows + 8) * b.abs()) @ w.abs()) * 1.01 \
            + u * val["gx"][has].abs() * 1.01 + small
        val["gt"] = scale * b.T @ y
        tol["gt"] = scale * ((b_off + E * (len(came) + 8) * b.abs()).T @ y.abs()) * 1.01 \
            + u * val["gt"].abs() * 1.01 + small
    return {n: (val[n], tol[n]) for n in val}
