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
        # rounded to the type: of up to 256 tokens in two parts
        b_off = p * g.abs()[:, None] * r + b.abs() * ((u if t > 256 else u * u) + 4 * E)
        # an exponential under float32's smallest normal number is 0, and so is its product under it:
        # off by at most that number, and by it times grad
        b_off = b_off + 2.0 ** -126 * (1 + g.abs()[:, None])
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


# -------------------------------------------------------- attention with decay --

def decay_attend(q, k, v, decay, at, scale, state=None, reverse=False, grad=None, grad_state=None):
    """{"out", "last" and with grad "gq", "gk", "gv", "gs"}: (value, bound)."""
    u = unit(q.dtype)
    heads, width = q.shape[1:]
    share, docs = heads // k.shape[1], len(at) - 1
    shape = (docs, heads, width, width)
    zeros = torch.zeros(shape, dtype=torch.float64)
    s0 = zeros if state is None else state.double()
    val = {"out": torch.zeros(q.shape, dtype=torch.float64), "last": s0.clone()}
    if grad is not None:
        b0 = zeros if grad_state is None else grad_state.double()
        val.update({n: torch.zeros(x.shape, dtype=torch.float64) for n, x in (("gq", q), ("gk", k), ("gv", v))})
        val["gs"] = b0.clone()
    tol = {n: torch.zeros_like(x) for n, x in val.items()}
    for d in range(docs):
        n = at[d + 1] - at[d]
        rows = torch.arange(at[d], at[d + 1])
        if reverse:
            rows = rows.flip(0)
        i = torch.arange(n, dtype=torch.float64)
        for h in range(heads):
            r, g = float(decay[h]), h // share
            x, y, z = q[rows, h].double(), k[rows, g].double(), v[rows, g].double()
            apart = i[:, None] - i[None]
            w = torch.where(apart >= 0, torch.exp(-r * apart.clamp(min=0)), 0.0)
            since, until, all_ = torch.exp(-r * (i + 1)), torch.exp(-r * (n - 1 - i)), math.exp(-r * n)
            # Of a weight: its exponent's roundings, and one for each chunk passed; of a sum: one
            # for each term and each product of `width`. Weights that small no longer count
            # are covered by the smallest normal number of the end.
            slack = E * (4 * r * n * (r * n < 100) + 400 * (r * n >= 100) + 2 * n + 2 * width + 80)
            # what fp16 drops under the largest of a product's operand: 2^-24 of it
            drop = 2.0 ** -23 if q.dtype == torch.float16 else 0.0

            def add(name, where, value, size, rel, low=0.0):
                val[name][where] += value
                tol[name][where] += size * (rel + slack) * 1.05 + low

            def low(a, b, c):
                """Dropped bits, where a row of |a| meets sums of |b| by |c| over n tokens or a state."""
                if not drop or not n:
                    return 0.0
                top = lambda t: float(t.abs().max()) if t.numel() else 0.0
                return 3 * drop * width * top(a) * top(b) * top(c) * float(w.sum(1).max() + 32)

            # A state's copy is rounded once. Weights within 32 tokens, and what enters a state, are in
            # parts of u^2 and less: documents of up to 32 tokens without a state round no copy.
            def parts(state):
                return 2 * u * u if n <= 32 and not state.any() else u + 2 * u * u

            S, S_abs = s0[d, h], s0[d, h].abs()
            s_low = drop * width * float(S_abs.max()) if drop else 0.0
            top = lambda t: float(t.abs().max()) if t.numel() else 0.0
            add("out", (rows, h), scale * ((w * (x @ y.T)) @ z + since[:, None] * (x @ S)),
                scale * ((w * (x.abs() @ y.abs().T)) @ z.abs() + since[:, None] * (x.abs() @ S_abs)), parts(S),
                scale * (low(x, y, z) + s_low * top(x)))
            val["last"][d, h] = all_ * S + (until[:, None] * y).T @ z
            tol["last"][d, h] = (all_ * S_abs + (until[:, None] * y.abs()).T @ z.abs()) * (slack + 8 * E) \
                + (2.0 ** -24 * top(y) * top(z) * float(until.sum()) if drop else 0.0)
            if grad is None:
                continue
            b = grad[rows, h].double()
            B, B_abs = b0[d, h], b0[d, h].abs()
            b_low = drop * width * float(B_abs.max()) if drop else 0.0
            add("gq", (rows, h), scale * ((w * (b @ z.T)) @ y + since[:, None] * (b @ S.T)),
                scale * ((w * (b.abs() @ z.abs().T)) @ y.abs() + since[:, None] * (b.abs() @ S_abs.T)), parts(S),
                scale * (low(b, z, y) + s_low * top(b)))
            add("gk", (rows, g), scale * (w * (b @ z.T)).T @ x + until[:, None] * (z @ B.T),
                scale * (w * (b.abs() @ z.abs().T)).T @ x.abs() + until[:, None] * (z.abs() @ B_abs.T), parts(B),
                scale * low(z, b, x) + b_low * top(z))
            add("gv", (rows, g), scale * (w * (x @ y.T)).T @ b + until[:, None] * (y @ B),
                scale * (w * (x.abs() @ y.abs().T)).T @ b.abs() + until[:, None] * (y.abs() @ B_abs), parts(B),
                scale * low(y, x, b) + b_low * top(y))
            val["gs"][d, h] = all_ * B + scale * (since[:, None] * x).T @ b
            tol["gs"][d, h] = (all_ * B_abs + scale * (since[:, None] * x.abs()).T @ b.abs()) * (slack + 8 * E) \
                + (2.0 ** -24 * scale * top(x) * top(b) * float(since.sum()) if drop else 0.0)
    small = torch.finfo(q.dtype).smallest_normal
    for name in tol:
        if name in ("last", "gs"):
            tol[name] = tol[name] + torch.finfo(torch.float32).smallest_normal
        else:
            tol[name] = tol[name] + u * val[name].abs() * 1.05 + small
    return {n: (val[n], tol[n]) for n in val}
