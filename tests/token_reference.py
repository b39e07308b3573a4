"""The token operators from their definitions, in 64 bits on the CPU, with a
bound on what a kernel that follows include/tokens.h may differ by.

Bounds count roundings: `u` is half a step of the tensors' type
(finfo.eps / 2), E that of float32. Each result comes with the largest error
that its roundings can add up to, to first order.
"""
import math

import torch

E = 2.0 ** -24


def unit(dtype):
    return torch.finfo(dtype).eps / 2


def check(got, want, bound, what):
    """|got - want| <= bound, elementwise, and no NaN where none is wanted."""
    got = got.detach().cpu().double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    off = (got - want).abs()
    bad = ~(off <= bound)
    if bad.any():
        at = tuple(int(i) for i in bad.nonzero()[0])
        worst = float((off / bound.clamp(min=1e-300)).nan_to_num(1e30).max())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {at}: got "
                             f"{float(got[at])!r}, want {float(want[at])!r}, bound "
                             f"{float(bound[at]):.3e}; worst {worst:.2f} of its bound")


# ------------------------------------------------------------------ embedding --

def embed(table, ids, scale):
    rows = table.shape[0]
    i = ids.reshape(-1).long()
    kept = (i >= 0) & (i < rows)
    out = torch.zeros((i.numel(), table.shape[1]), dtype=torch.float64)
    out[kept] = table.double()[i[kept]] * scale
    out = out.reshape(*ids.shape, table.shape[1])
    # the product in float32, then the type; half a step of the smallest number under it
    return out, out.abs() * (unit(table.dtype) + 2 * E) + torch.finfo(table.dtype).smallest_normal


def embed_grad(grad, ids, rows, scale):
    g, i = grad.reshape(-1, grad.shape[-1]).double(), ids.reshape(-1).long()
    kept = (i >= 0) & (i < rows)
    total, size = (torch.zeros((rows, g.shape[1]), dtype=torch.float64) for _ in range(2))
    total.index_add_(0, i[kept], g[kept])
    size.index_add_(0, i[kept], g[kept].abs())
    terms = torch.bincount(i[kept], minlength=rows)[:, None].double()
    total, size = total * scale, size * abs(scale)
    # a sum of n terms in any order: at most n - 1 roundings on a term; the scale's product: 2
    bound = size * (terms + 2) * E + total.abs() * unit(grad.dtype)
    return total, bound + torch.finfo(grad.dtype).smallest_normal


# ------------------------------------------------------------------ attention --

def attend(q, k, v, q_at, k_at, scale, cap=0.0, slopes=None, q_pos=None, k_pos=None, causal=False,
           prefix=None, grad=None):
    """{"out": (value, bound), "lse": ..., and with grad "gq", "gk", "gv"}."""
    u = unit(q.dtype)
    heads, width = q.shape[1:]
    share = heads // k.shape[1]
    made = {"out": q, "lse": q[:, :, 0]}
    if grad is not None:
        made.update(gq=q, gk=k, gv=v)
    val = {n: torch.zeros(t.shape, dtype=torch.float64) for n, t in made.items()}
    tol = {n: torch.zeros(t.shape, dtype=torch.float64) for n, t in made.items()}
    val["lse"].fill_(-math.inf)
    for d in range(len(q_at) - 1):
        qs, ks = slice(q_at[d], q_at[d + 1]), slice(k_at[d], k_at[d + 1])
        lq, lk = q_at[d + 1] - q_at[d], k_at[d + 1] - k_at[d]
        if lq == 0 or lk == 0:
            continue
        i, j = torch.arange(lq)[:, None], torch.arange(lk)[None]
        seen = torch.ones((lq, lk), dtype=torch.bool)
        if causal or prefix is not None:
            seen = j <= i + (lk - lq)
            if prefix is not None:
                seen = seen | (j < int(prefix[d]))
        some = seen.any(1)
        for h in range(heads):
            x, y, w = q[qs, h].double(), k[ks, h // share].double(), v[ks, h // share].double()
            s = x @ y.T * scale
            off = E * (width + 8) * scale * (x.abs() @ y.abs().T)  # a product of `width` terms
            flat, z = torch.ones_like(s), s
            if cap:
                flat = 1 - torch.tanh(s / cap) ** 2
                z = cap * torch.tanh(s / cap)
                off = off + E * (16 * cap + 8 * s.abs())  # exp, sum, quotient, product, difference
            if slopes is not None:
                far = (q_pos[qs].double()[:, None] - k_pos[ks].double()[None]).abs().sum(2)
                z = z - float(slopes[h]) * far
                off = off + 4 * E * float(slopes[h]) * far
            off = off + 8 * E * (z.abs() + 1)
            z = z.masked_fill(~seen, -math.inf)
            lse = torch.logsumexp(z, 1).masked_fill(~some, -math.inf)
            p = torch.exp(z - lse[:, None]).masked_fill(~seen, 0.0)
            # a weight's relative error: its score's, the sum's of lk terms and their scores'
            off = off + E * (lse.abs().nan_to_num(0, 0, 0)[:, None] * 4 + 8)
            r = off + (p * off).sum(1, keepdim=True) + E * (lk + 16)
            val["lse"][qs, h] = lse
            tol["lse"][qs, h] = ((p * off).sum(1) + E * (lk + 16)) + E * lse.abs().nan_to_num(0, 0, 0) * 4
            out = p @ w
            # each weight is rounded, in the product and perhaps in the sum
            out_off = (p * (2 * u + r + E * lk)) @ w.abs()
            val["out"][qs, h], tol["out"][qs, h] = out, out_off + u * out.abs()
            if grad is None:
                continue
            g = grad[qs, h].double()
            dp = g @ w.T
            dp_off = E * (width + 8) * (g.abs() @ w.abs().T)
            delta = (p * dp).sum(1, keepdim=True)
            delta_off = (p * (dp_off + dp.abs() * (r + E * (lk + width)))).sum(1, keepdim=True) \
                + delta.abs() * r.amax(1, keepdim=True)
            ds = p * (dp - delta) * flat
            bend = 16 * E * (1 + s.abs() / cap) if cap else 0.0
            ds_off = ds.abs() * (u + r + 8 * E) + p * flat * (dp_off + delta_off) \
                + p * (dp - delta).abs() * bend
            # grad_q starts from the rounded output's delta, corrected after its products
            first = (g.abs() * (out_off + u * out.abs())).sum(1, keepdim=True)
            gq_off = ds_off + 2 * u * p * flat * first
            val["gq"][qs, h] = scale * ds @ y
            tol["gq"][qs, h] = scale * ((gq_off + E * (lk + 8) * ds.abs()) @ y.abs()) \
                + u * val["gq"][qs, h].abs()
            n = lq * share
            val["gk"][ks, h // share] += scale * ds.T @ x
            tol["gk"][ks, h // share] += scale * ((ds_off + E * (n + 8) * ds.abs()).T @ x.abs())
            val["gv"][ks, h // share] += p.T @ g
            tol["gv"][ks, h // share] += (p * (u + r + E * (n + 8))).T @ g.abs()
    small = torch.finfo(q.dtype).smallest_normal
    for n in ("gk", "gv"):
        if n in tol:
            tol[n] += u * val[n].abs()
    for n in tol:
        if n != "lse":
            tol[n] = tol[n] * 1.01 + small
    return {n: (val[n], tol[n]) for n in val}


# ----------------------------------------------------------------- recurrence --

def scan(gate, x, at, state=None, reverse=False, grad=None, grad_state=None):
    """{"y", "last" and with grad "gg", "gx", "gs"}: (value, bound)."""
    u = unit(x.dtype)
    docs, width = len(at) - 1, x.shape[1]
    f, z = gate.double(), x.double()
    a, keep = torch.sigmoid(f), torch.sigmoid(-f)
    # both gates are right to a few roundings: of the exponent's argument and of its function
    rel = E * (f.abs() + 8)
    zeros = torch.zeros((docs, width), dtype=torch.float64)
    h0 = zeros if state is None else state.double()
    val = {"y": torch.zeros_like(z), "last": h0.clone()}
    tol = {n: torch.zeros_like(t) for n, t in val.items()}
    before, b_off, size = (torch.zeros_like(z) for _ in range(3))
    orders = [list(range(b, e))[::-1 if reverse else 1] for b, e in zip(at[:-1], at[1:])]
    for d, order in enumerate(orders):
        h, off, n = h0[d], torch.zeros(width, dtype=torch.float64), h0[d].abs()
        for t in order:
            before[t], b_off[t] = h, off
            h = a[t] * h + keep[t] * z[t]
            # products of gates over a chunk carry the same roundings, and two more each
            off = a[t] * off + 2 * (rel[t] + 3 * E) * (a[t] * n + keep[t] * z[t].abs())
            n = a[t] * n + keep[t] * z[t].abs()
            val["y"][t], tol["y"][t] = h, off + u * h.abs()
        val["last"][d], tol["last"][d] = h, off
    if grad is not None:
        g0 = zeros if grad_state is None else grad_state.double()
        val.update(gg=torch.zeros_like(z), gx=torch.zeros_like(z), gs=g0.clone())
        tol.update(gg=torch.zeros_like(z), gx=torch.zeros_like(z), gs=torch.zeros_like(g0))
        g = grad.double()
        for d, order in enumerate(orders):
            back, off, n = g0[d], torch.zeros(width, dtype=torch.float64), g0[d].abs()
            for t in reversed(order):
                dh, n = back + g[t], n + g[t].abs()
                d_off = off + 2 * E * n
                k = before[t] - z[t]
                val["gg"][t] = dh * k * a[t] * keep[t]
                tol["gg"][t] = a[t] * keep[t] * (
                    d_off * k.abs() + dh.abs() * (b_off[t] + 2 * E * k.abs())
                    + dh.abs() * k.abs() * (2 * rel[t] + 6 * E)) + u * val["gg"][t].abs()
                val["gx"][t] = dh * keep[t]
                tol["gx"][t] = d_off * keep[t] + (rel[t] + 2 * E + u) * val["gx"][t].abs()
                back = dh * a[t]
                off = a[t] * d_off + 2 * (rel[t] + 3 * E) * a[t] * n
                n = a[t] * n
            val["gs"][d], tol["gs"][d] = back, off
    for n in tol:
        # 0 * 0 of the exponent's smallest results; two chunked orders of the sum
        tol[n] = 2 * tol[n] - u * val[n].abs() * (n in ("y", "gg", "gx")) \
            + torch.finfo(x.dtype).smallest_normal
    return {n: (val[n], tol[n]) for n in val}
