"""Operators of a model that predicts pillar tokens: rotary positions, attention with decay, and the
loss over the rows of a table.

A model that goes through a frame's pillars (or a scan's points) in order and says which cell comes
next turns its queries and keys by their places on the grid, mixes the tokens at a cost that grows
with their number alone, and compares every token's output with the learned rows of all cells. Each
operator is here in its plain form (elementary torch operations in 32 bits, rounded once at the end;
angles in 64) and as the framework's call, over the same inputs.

  rotate       pairs of a head's elements turned by position * frequency, the rest of the head kept
  decay        S[t] = exp(-decay) S[t-1] + k[t] v[t]^T per head, out[t] = scale * q[t] S[t]
  decay_train  the same, then the gradients of q, k, v and the initial state
  loss         log sum over rows of exp(scale * x.row), less scale * x.table[ids[i]]
  loss_train   the same, then the gradients of x and the table
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
GRID = (496, 432)  # pillar rows and columns of the 0.16 m grid
CELLS = GRID[0] * GRID[1]


def listed():
    return [
        # queries and keys of one new token in each of 64 sequences, 16 heads and 4 key heads: latency
        {"name": "rotate_token", "op": "rotate", "dtype": "bf16", "tokens": 64, "heads": 20,
         "width": 128, "rotated": 128, "axes": 1, "far": 12000, "interleaved": False,
         "inverse": False, "stretch": 1.0, "context": 0},
        # queries and keys of a frame's points, turned by their row and column on the grid
        {"name": "rotate_points", "op": "rotate", "dtype": "bf16", "tokens": 122880, "heads": 10,
         "width": 128, "rotated": 128, "axes": 2, "far": 0, "interleaved": False, "inverse": False,
         "stretch": 1.0, "context": 0},
        # gradients of a training step turned back: a quarter of the head, far into a long scan whose
        # frequencies are scaled for it
        {"name": "rotate_long_grad", "op": "rotate", "dtype": "fp32", "tokens": 30011, "heads": 8,
         "width": 80, "rotated": 20, "axes": 1, "far": 1000000, "interleaved": True, "inverse": True,
         "stretch": 32.0, "context": 12000},
        # one new token in each of 64 sequences: every state is read, changed and used once
        {"name": "decay_token", "op": "decay", "dtype": "bf16", "docs": 64, "length": 1, "ragged": 0.0,
         "heads": 16, "kv_heads": 4, "width": 128, "state": True, "keep": False, "reverse": False},
        # sixteen frames of pillars in scan order, forward only, from no state
        {"name": "decay_frames", "op": "decay", "dtype": "bf16", "docs": 16, "length": 12000,
         "ragged": 0.3, "heads": 8, "kv_heads": 8, "width": 64, "state": False, "keep": False,
         "reverse": False},
        # a training step over the points of one frame, too many to attend to each other
        {"name": "decay_points_train", "op": "decay_train", "dtype": "bf16", "docs": 1,
         "length": 122880, "ragged": 0.0, "heads": 8, "kv_heads": 8, "width": 128, "state": True,
         "keep": False, "reverse": False},
        # a training step over windows of a few dozen voxels each, shared key heads
        {"name": "decay_windows_train", "op": "decay_train", "dtype": "fp16", "docs": 500,
         "length": 36, "ragged": 1.0, "heads": 8, "kv_heads": 2, "width": 32, "state": False,
         "keep": True, "reverse": True},
        # how likely the next cell was, for one token of each of 16 sequences
        {"name": "loss_token", "op": "loss", "dtype": "bf16", "tokens": 16, "rows": CELLS,
         "width": 256, "scale": 1.0},
        # how likely each cell of a frame at the voxel budget was
        {"name": "loss_frame", "op": "loss", "dtype": "bf16", "tokens": 12000, "rows": CELLS,
         "width": 128, "scale": 2.0},
        # a training step over frames, every cell a row
        {"name": "loss_frames_train", "op": "loss_train", "dtype": "bf16", "tokens": 4096,
         "rows": CELLS, "width": 512, "scale": 1.0},
        # a training step of a small model over a coarse grid, odd everywhere
        {"name": "loss_coarse_train", "op": "loss_train", "dtype": "fp16", "tokens": 997,
         "rows": 13391, "width": 96, "scale": 1.0},
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    hi = max(lo, hi)
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rotate", "decay", "decay_train", "loss", "loss_train"])
    if op == "rotate":
        heads, width = rng.choice([1, 3, 8, 10, 20]), rng.choice([32, 48, 64, 80, 100, 128])
        axes = rng.choice([1, 1, 2, 3])
        pairs = rng.choice([width // (2 * axes), width // (4 * axes), rng.randint(1, width // (2 * axes))])
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        size = DTYPES[dtype].itemsize
        return {"op": op, "dtype": dtype, "tokens": _between(rng, 1, 122880 * 2560 // (heads * width * size)),
                "heads": heads, "width": width, "rotated": 2 * axes * pairs, "axes": axes,
                "far": 0 if axes > 1 else rng.choice([12000, 122880, 1000000]),
                "interleaved": rng.random() < 0.5, "inverse": rng.random() < 0.5,
                "stretch": rng.choice([1.0, 4.0, 32.0]), "context": rng.choice([0, 12000])}
    if op in ("decay", "decay_train"):
        kv_heads = rng.choice([1, 2, 4, 8])
        heads = kv_heads * rng.choice([g for g in (1, 1, 2, 4) if g * kv_heads <= 16])
        width = rng.choice([32, 48, 64, 96, 128])
        docs = _between(rng, 1, min(500, (1 << 26) // (heads * width * width)))
        t = 122880 * 1024 // (heads * width)
        return {"op": op, "dtype": rng.choice(["bf16", "fp16"]), "docs": docs,
                "length": rng.choice([1, _between(rng, 1, min(122880, t // docs))]) if op == "decay"
                else _between(rng, 1, min(122880, t // docs)),
                "ragged": rng.choice([0.0, 0.3, 1.0]), "heads": heads, "kv_heads": kv_heads,
                "width": width, "state": rng.random() < 0.5, "keep": rng.random() < 0.3,
                "reverse": rng.random() < 0.3}
    width = rng.choice([32, 64, 72, 128, 200, 256, 512, 1000])
    rows = _between(rng, 100, CELLS)
    most = min(12000, 4096 * CELLS * 512 // (rows * width))
    return {"op": op, "dtype": rng.choice(["bf16", "fp16"]), "tokens": _between(rng, 1, most),
            "rows": rows, "width": width, "scale": rng.choice([0.5, 1.0, 3.0])}


def _lengths(case):
    """Lengths of a case's documents: `length`, less up to `ragged` of it; the first is whole."""
    docs, length = case["docs"], case["length"]
    u = torch.rand(docs, generator=torch.Generator().manual_seed(docs), dtype=torch.float64)
    u[0] = 0.0
    return [int(v) for v in (length - torch.floor(u * (case["ragged"] * length))).tolist()]


def _normal(shape, gen, dtype, std=1.0):
    return (torch.randn(shape, generator=gen, device=gen.device) * std).to(dtype)


def _frequencies(case):
    """Radians per position of each axis and pair, in 64 bits on the host: base ** (-pair / pairs),
    and where a context is stretched, slow pairs divided by as much, those that turn more than 32
    times within the context kept, and those between 1 and 32 turns between the two."""
    pairs = case["rotated"] // (2 * case["axes"])
    f = 10000.0 ** (-np.arange(pairs) / pairs)
    if case["stretch"] != 1.0:
        kept = 0.0
        if case["context"]:
            kept = np.clip((case["context"] * f / (2 * math.pi) - 1.0) / 31.0, 0.0, 1.0)
        f = f * ((1.0 - kept) / case["stretch"] + kept)
    return torch.from_numpy(np.tile(f, (case["axes"], 1)))


def prepare(case, seed):
    device = torch.device("cuda")
    gen = torch.Generator(device=device).manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    s = dict(case)
    if case["op"] == "rotate":
        t, axes = case["tokens"], case["axes"]
        s["x"] = _normal((t, case["heads"], case["width"]), gen, dtype)
        top = [case["far"]] if case["far"] else [40, *GRID][-axes:]
        u = torch.rand((t, axes), generator=gen, device=device, dtype=torch.float64)
        s["pos"] = (u * torch.tensor(top, device=device)).to(torch.int32)
        if own:
            import sparse_spatial_hashing_amd as ssh
            s["freqs"] = ssh.rotary_frequencies(case["rotated"], axes=axes, stretch=case["stretch"],
                                                context=case["context"], device=device)
        else:
            s["freqs"] = _frequencies(case).to(device)
        return s
    if case["op"] in ("decay", "decay_train"):
        heads, kv_heads, width, docs = case["heads"], case["kv_heads"], case["width"], case["docs"]
        lens = _lengths(case)
        t = sum(lens)
        s["most"] = max(lens)
        s["offsets"] = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32).to(device)
        s["q"] = _normal((t, heads, width), gen, dtype)
        s["k"] = _normal((t, kv_heads, width), gen, dtype)
        s["v"] = _normal((t, kv_heads, width), gen, dtype)
        s["scale"] = 1.0 / math.sqrt(width)
        # heads that forget within ten tokens to within a few thousand; the first may forget nothing
        s["decay"] = torch.pow(2.0, -3.0 - 9.0 * torch.arange(heads, device=device) / heads)
        if case["keep"]:
            s["decay"][0] = 0.0
        shape = (docs, heads, width, width)
        s["state0"] = _normal(shape, gen, torch.float32, 4.0) if case["state"] else None
        if case["op"] == "decay_train":
            s["grad"] = _normal((t, heads, width), gen, dtype)
            s["grad_state"] = _normal(shape, gen, torch.float32) if case["state"] else None
        return s
    t, rows, width = case["tokens"], case["rows"], case["width"]
    s["table"] = _normal((rows, width), gen, dtype, 1.0 / math.sqrt(width))
    ids = torch.randint(0, rows, (t,), generator=gen, device=device)
    x = torch.randn((t, width), generator=gen, device=device)
    # the row that came is likelier by some, and one token in twelve (a frame's last) has none
    s["x"] = (x + 4.0 * s["table"][ids].float()).to(dtype)
    s["ids"] = torch.where(torch.rand(t, generator=gen, device=device) < 1 / 12, -1, ids)
    if case["op"] == "loss_train":
        # about the mean's weights; in fp16 as a scaled loss has them
        up = 1024.0 if case["dtype"] == "fp16" else 1.0
        s["grad"] = (torch.rand(t, generator=gen, device=device) + 0.5) * (up / t)
    return s


# ---------------------------------------------------------------------------------- plain forms --

def _rotate(s):
    x, rotated, axes = s["x"].float(), s["rotated"], s["axes"]
    angle = s["pos"].double()[:, :, None] * s["freqs"]  # [tokens, axes, pairs]
    if s["inverse"]:
        angle = -angle
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    part = x[:, :, :rotated].unflatten(2, (axes, -1))
    if s["interleaved"]:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], 4)
    else:
        a, b = part.chunk(2, 3)
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], 3)
    return torch.cat([turned.flatten(2), x[:, :, rotated:]], 2).to(s["x"].dtype)


_PART = 256  # tokens that see each other by their scores; the ones before by the state


class _Documents:
    """Packed rows as [docs, heads, parts, _PART, width] in 32 bits, and back."""

    def __init__(self, s):
        at = torch.arange(-(-s["most"] // _PART) * _PART, device=s["q"].device)
        self.offsets, self.total, self.heads = s["offsets"], s["q"].shape[0], s["heads"]
        lens = self.offsets[1:] - self.offsets[:-1]
        self.lens, self.there, self.reverse = lens, at[None] < lens[:, None], s["reverse"]
        turn = lens[:, None] - 1 - at[None] if s["reverse"] else at[None].expand(len(lens), -1)
        self.rows = torch.where(self.there, self.offsets[:-1, None] + turn, 0).long()
        # tokens of each part, and each token's distance to its part's end
        self.filled = self.there.unflatten(1, (-1, _PART)).sum(2)

    def split(self, x):
        x = torch.where(self.there[:, :, None, None], x[self.rows].float(), 0.0).transpose(1, 2)
        x = x.repeat_interleave(self.heads // x.shape[1], 1)
        return x.unflatten(2, (-1, _PART)).contiguous()

    def join(self, x):
        x = x.flatten(2, 3).transpose(1, 2)
        at = torch.arange(self.total, device=x.device)
        doc = torch.searchsorted(self.offsets[1:], at, right=True)
        at = at - self.offsets[doc]
        if self.reverse:
            at = self.lens[doc] - 1 - at
        return x[doc, at]


def _decay(s):
    docs = _Documents(s)
    q, k, v = docs.split(s["q"]), docs.split(s["k"]), docs.split(s["v"])
    rate = s["decay"][None, :, None]
    i = torch.arange(_PART, device=q.device)
    apart = (i[:, None] - i[None]).float()
    seen = torch.where(apart >= 0, torch.exp(-rate[..., None] * apart.clamp(min=0)), 0.0)  # [1, heads, i, j]
    entering = torch.exp(-rate * (i + 1))[..., None]  # of the state, at each token of a part
    left = (docs.filled[:, None, :, None] - 1 - i).clamp(min=0)  # [docs, 1, parts, i]: steps to the part's end
    leaving = torch.exp(-rate[..., None] * left)[..., None]
    through = torch.exp(-rate * docs.filled[:, None])[..., None, None]  # [docs, heads, parts, 1, 1]
    state = s["state0"]
    if state is None:
        state = torch.zeros((q.shape[0], s["heads"], s["width"], s["width"]), device=q.device)
    out, states = torch.empty_like(q), []
    for p in range(q.shape[2]):
        states.append(state)
        scores = torch.matmul(q[:, :, p], k[:, :, p].transpose(2, 3).contiguous()) * seen
        out[:, :, p] = s["scale"] * (torch.matmul(scores, v[:, :, p])
                                     + entering * torch.matmul(q[:, :, p], state))
        fresh = (k[:, :, p] * leaving[:, :, p]).transpose(2, 3).contiguous()
        state = through[:, :, p] * state + torch.matmul(fresh, v[:, :, p])
    made = docs.join(out).to(s["q"].dtype)
    if s["op"] == "decay":
        return made, state
    g = docs.split(s["grad"]) * s["scale"]
    back = s["grad_state"]
    if back is None:
        back = torch.zeros_like(state)
    gq, gk, gv = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
    for p in reversed(range(q.shape[2])):
        gp, kp, vp, qp = g[:, :, p], k[:, :, p], v[:, :, p], q[:, :, p]
        weights = torch.matmul(qp, kp.transpose(2, 3).contiguous()) * seen
        back_weights = torch.matmul(gp, vp.transpose(2, 3).contiguous()) * seen
        gq[:, :, p] = torch.matmul(back_weights, kp) \
            + entering * torch.matmul(gp, states[p].transpose(2, 3).contiguous())
        gk[:, :, p] = torch.matmul(back_weights.transpose(2, 3).contiguous(), qp) \
            + leaving[:, :, p] * torch.matmul(vp, back.transpose(2, 3).contiguous())
        gv[:, :, p] = torch.matmul(weights.transpose(2, 3).contiguous(), gp) \
            + leaving[:, :, p] * torch.matmul(kp, back)
        back = through[:, :, p] * back \
            + torch.matmul((qp * entering).transpose(2, 3).contiguous(), gp)
    gq, gk, gv = docs.join(gq), docs.join(gk), docs.join(gv)
    shared = (gk.shape[0], s["kv_heads"], -1, s["width"])
    made = (made, gq.to(s["q"].dtype), gk.view(shared).sum(2).to(s["k"].dtype),
            gv.view(shared).sum(2).to(s["v"].dtype))
    return (*made, state, back) if s["state0"] is not None else made


_PIECE = 16384  # rows of the table whose logits are held at once


def _loss(s):
    x, table, ids = s["x"].float(), s["table"], s["ids"]
    kept = (ids >= 0) & (ids < s["rows"])
    top = torch.full((x.shape[0],), -math.inf, device=x.device)
    total = torch.zeros_like(top)
    pieces = [slice(b, min(b + _PIECE, s["rows"])) for b in range(0, s["rows"], _PIECE)]
    for at in pieces:
        z = torch.matmul(x, table[at].float().t().contiguous()) * s["scale"]
        new = torch.maximum(top, z.amax(1))
        total = total * torch.exp(top - new) + torch.exp(z - new[:, None]).sum(1)
        top = new
    lse = top + torch.log(total)
    came = ids.clamp(0, s["rows"] - 1)
    loss = torch.where(kept, lse - s["scale"] * (x * table[came].float()).sum(1), 0.0)
    if s["op"] == "loss":
        return loss
    by = torch.where(kept, s["grad"], 0.0) * s["scale"]
    gx = torch.zeros_like(x)
    gt = torch.empty((s["rows"], s["width"]), device=x.device)
    for at in pieces:
        part = table[at].float()
        p = torch.exp(torch.matmul(x, part.t().contiguous()) * s["scale"] - lse[:, None])
        inside = ((came >= at.start) & (came < at.stop)).nonzero()[:, 0]
        p[inside, came[inside] - at.start] -= 1.0
        p *= by[:, None]
        gx += torch.matmul(p, part)
        gt[at] = torch.matmul(p.t().contiguous(), x)
    return loss, gx.to(s["x"].dtype), gt.to(table.dtype)


# ------------------------------------------------------------------------------ the framework's --

def _own(s):
    import sparse_spatial_hashing_amd as ssh
    if s["op"] == "rotate":
        return ssh.rotate(s["x"], s["pos"], s["freqs"], interleaved=s["interleaved"], inverse=s["inverse"])
    if s["op"] in ("decay", "decay_train"):
        more = dict(state=s["state0"], scale=s["scale"], reverse=s["reverse"])
        if s["op"] == "decay":
            return ssh.decay_attend(s["q"], s["k"], s["v"], s["decay"], s["offsets"], **more)
        whole = s["state0"] is not None
        out, state, carry = ssh.decay_attend(s["q"], s["k"], s["v"], s["decay"], s["offsets"],
                                             return_state=whole, return_carry=True, **more)
        gq, gk, gv, gs = ssh.decay_attend_grad(s["grad"], s["q"], s["k"], s["v"], s["decay"], carry,
                                               s["offsets"], grad_state=s["grad_state"], **more)
        return (out, gq, gk, gv, state, gs) if whole else (out, gq, gk, gv)
    if s["op"] == "loss":
        return ssh.row_loss(s["x"], s["table"], s["ids"], scale=s["scale"])
    loss, lse = ssh.row_loss(s["x"], s["table"], s["ids"], scale=s["scale"], return_lse=True)
    return (loss, *ssh.row_loss_grad(s["grad"], s["x"], s["table"], s["ids"], lse, scale=s["scale"]))


def run(state):
    if own:
        return _own(state)
    op = state["op"].replace("_train", "")
    return {"rotate": _rotate, "decay": _decay, "loss": _loss}[op](state)


# ---------------------------------------------------------------------------- work and 64 bits --

def work(case):
    size = DTYPES[case["dtype"]].itemsize
    op = case["op"]
    if op == "rotate":
        t, elements = case["tokens"], case["tokens"] * case["heads"] * case["width"]
        return {"bytes": 2 * elements * size + 4 * t * case["axes"],
                "flops": 3 * t * case["heads"] * case["rotated"]}
    if op in ("decay", "decay_train"):
        heads, kv_heads, width, docs = case["heads"], case["kv_heads"], case["width"], case["docs"]
        t, train = sum(_lengths(case)), op == "decay_train"
        state = docs * heads * width * width * 4
        rows = t * (heads + kv_heads) * width * size * (4 if train else 2)
        if train:
            state = state * 4 if case["state"] else 0  # states and their gradients
        else:
            state = state * 2 if case["state"] else state
        # a token meets its document by a state of width x width, or its tokens if they are fewer
        inner = min(width, t / docs)
        return {"bytes": rows + state, "flops": (12 if train else 4) * t * heads * width * inner}
    t, rows, width = case["tokens"], case["rows"], case["width"]
    train = op == "loss_train"
    # the logits are not kept: their product is taken again before the gradients' two
    return {"bytes": (t + rows) * width * size * (2 if train else 1) + 12 * t,
            "flops": (8 if train else 2) * t * rows * width}


def _exact_rotate(s):
    """Pairs as complex numbers, multiplied by the angle's."""
    axes, rotated = s["axes"], s["rotated"]
    pairs = rotated // (2 * axes)
    x = s["x"].double()
    out = x.clone()
    sign = -1.0 if s["inverse"] else 1.0
    f = _frequencies(s)[0].to(x.device)
    for axis in range(axes):
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device).expand(x.shape[0], pairs),
                           sign * s["pos"][:, axis, None].double() * f)[:, None]
        at = torch.arange(pairs, device=x.device)
        first = 2 * pairs * axis + (2 * at if s["interleaved"] else at)
        second = first + (1 if s["interleaved"] else pairs)
        z = torch.complex(x[:, :, first], x[:, :, second]) * turn
        out[:, :, first], out[:, :, second] = z.real, z.imag
    return out


def _exact_decay(s):
    """Every pair of a document's tokens, by rows of them."""
    train = s["op"] == "decay_train"
    share, scale, at = s["heads"] // s["kv_heads"], s["scale"], s["offsets"].tolist()
    device = s["q"].device
    made = [torch.zeros(s[n].shape, dtype=torch.float64, device=device)
            for n in (("q", "q", "k", "v") if train else ("q",))]
    shape = (s["docs"], s["heads"], s["width"], s["width"])
    last, first = (torch.zeros(shape, dtype=torch.float64, device=device) for _ in range(2))
    rate = s["decay"].double()
    for d in range(s["docs"]):
        rows, n = slice(at[d], at[d + 1]), at[d + 1] - at[d]
        turn = (lambda x: x.flip(0)) if s["reverse"] else (lambda x: x)
        step = torch.arange(n, device=device, dtype=torch.float64)
        for h in range(s["heads"]):
            r, kv = rate[h], h // share
            q, k, v = (turn(s[name][rows, j].double()) for name, j in (("q", h), ("k", kv), ("v", kv)))
            s0 = None if s["state0"] is None else s["state0"][d, h].double()
            since, until = torch.exp(-r * (step + 1))[:, None], torch.exp(-r * (n - 1 - step))[:, None]
            last[d, h] = (until * k).T @ v
            if s0 is not None:
                last[d, h] += torch.exp(-r * n) * s0
            out, gq, gk, gv = (torch.zeros_like(q) for _ in range(4))
            if train:
                g = turn(s["grad"][rows, h].double()) * scale
                s1 = None if s["grad_state"] is None else s["grad_state"][d, h].double()
            for b in range(0, n, 4096):
                e = min(n, b + 4096)
                fall = step[b:e, None] - step[None, :e]
                fall = torch.where(fall >= 0, torch.exp(-r * fall.clamp(min=0)), 0.0)
                w = (q[b:e] @ k[:e].T) * fall
                out[b:e] = w @ v[:e]
                if train:
                    back = (g[b:e] @ v[:e].T) * fall
                    gq[b:e] = back @ k[:e]
                    gk[:e] += back.T @ q[b:e]
                    gv[:e] += w.T @ g[b:e]
            if s0 is not None:
                out += since * (q @ s0)
            made[0][rows, h] = turn(out) * scale
            if not train:
                continue
            if s0 is not None:
                gq += since * (g @ s0.T)
                first[d, h] = (since * q).T @ g
            if s1 is not None:
                gk += until * (v @ s1.T)
                gv += until * (k @ s1)
                first[d, h] += torch.exp(-r * n) * s1
            made[1][rows, h] = turn(gq)
            made[2][rows, kv] += turn(gk)
            made[3][rows, kv] += turn(gv)
    if not train:
        return made[0], last
    return (*made, last, first) if s["state0"] is not None else tuple(made)


def _exact_loss(s):
    """Token by token against all rows, a few hundred at once."""
    train = s["op"] == "loss_train"
    table = s["table"].double() * s["scale"]
    loss = torch.zeros(s["tokens"], dtype=torch.float64, device=table.device)
    gx = torch.zeros(s["x"].shape, dtype=torch.float64, device=table.device)
    gt = torch.zeros_like(table)
    for b in range(0, s["tokens"], 512):
        x, ids = s["x"][b:b + 512].double(), s["ids"][b:b + 512]
        kept = ids >= 0
        logits = x @ table.T
        log_p = torch.log_softmax(logits, 1)
        loss[b:b + 512][kept] = -log_p[kept, ids[kept]]
        if train:
            back = torch.exp(log_p)
            back[kept, ids[kept]] -= 1.0
            back *= torch.where(kept, s["grad"][b:b + 512].double(), 0.0)[:, None]
            gx[b:b + 512] = back @ table
            gt += back.T @ x
    return (loss, gx, gt * s["scale"]) if train else loss


def exact(case, seed):
    if case["op"].startswith("decay"):
        pairs = sum(n * n + 4096.0 * 64 for n in _lengths(case)) * case["heads"] * case["width"]
        if pairs > 1.6e13 or case["docs"] * case["heads"] > 8000:
            return None
    s = prepare(case, seed)
    op = case["op"].replace("_train", "")
    return {"rotate": _exact_rotate, "decay": _exact_decay, "loss": _exact_loss}[op](s)
