"""Token operators on the GPU against their definitions in 64 bits."""
import itertools
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import sparse_spatial_hashing_amd as ssh  # noqa: E402
import token_reference as ref  # noqa: E402

DEV = torch.device("cuda:0")
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _ends(lens, first=0):
    return [first] + [first + n for n in itertools.accumulate(lens)]


def _at(ends):
    return torch.tensor(ends, dtype=torch.int32, device=DEV)


def _randn(shape, dtype, gen, std=1.0):
    return (torch.randn(shape, generator=gen) * std).to(dtype)


# ------------------------------------------------------------------ embedding --

@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("width", [1, 7, 32, 33, 100, 128, 250, 1032])
def test_embed(dtype, width):
    gen = torch.Generator().manual_seed(width)
    table = _randn((57, width), dtype, gen)
    for n, index in ((0, torch.int32), (1, torch.int64), (97, torch.int32), (613, torch.int64)):
        ids = torch.randint(-2, 60, (n,), generator=gen, dtype=index)
        print(f"embed {dtype} width {width} n {n}", flush=True)
        got = ssh.embed(table.to(DEV), ids.to(DEV), scale=1.75)
        ref.check(got, *ref.embed(table, ids, 1.75), "embed")
        g = _randn((n, width), dtype, gen)
        got = ssh.embed_grad(g.to(DEV), ids.to(DEV), 57, scale=1.75)
        assert got.dtype == dtype
        ref.check(got, *ref.embed_grad(g, ids, 57, 1.75), "embed_grad")


@pytest.mark.parametrize("n,rows,spread", [(5000, 3, 1.0), (20000, 1, 1.0), (64, 1, 1.0), (65, 2, 1.0),
                                           (40000, 100000, 3.0), (9000, 700, 1.0), (4097, 5000, 8.0),
                                           (130000, 60000, 2.0), (70000, 17, 1.0), (256, 130, 1.0),
                                           (255, 2, 1.0), (3, 100000, 1.0), (257, 65, 1.0)])
@pytest.mark.parametrize("width,dtype", [(8, F32), (64, BF16), (33, F16)])
def test_embed_grad_long_rows(n, rows, spread, width, dtype):
    """Rows with no token, one, and so many that they cross every border of the sum."""
    gen = torch.Generator().manual_seed(n + rows)
    ids = (torch.rand(n, generator=gen).double().pow(spread) * rows).long().clamp(max=rows - 1)
    ids[torch.rand(n, generator=gen) < 0.05] = -1
    g = _randn((n, width), dtype, gen)
    print(f"embed_grad n {n} rows {rows} width {width}", flush=True)
    one = ssh.embed_grad(g.to(DEV), ids.to(DEV), rows, scale=0.5)
    ref.check(one, *ref.embed_grad(g, ids, rows, 0.5), "embed_grad")
    assert torch.equal(one, ssh.embed_grad(g.to(DEV), ids.to(DEV), rows, scale=0.5))
    assert torch.equal(one, ssh.embed_grad(g.to(DEV), ids.int().to(DEV), rows, scale=0.5))


def test_embed_all_without_a_row():
    ids = torch.full((300,), -1, dtype=torch.int32, device=DEV)
    g = torch.full((300, 40), math.nan, device=DEV)
    assert not ssh.embed_grad(g, ids, 9).any()
    assert not ssh.embed(torch.full((9, 40), math.inf, device=DEV), ids).any()


def test_embed_strides_shapes_and_autograd():
    gen = torch.Generator().manual_seed(1)
    wide = _randn((40, 100), F32, gen).to(DEV)
    for table in (wide[:, 1:34], wide[::2, :64], wide.t()[:50], wide[3:, 4:36]):
        ids = torch.randint(-1, table.shape[0] + 1, (3, 17), generator=gen)
        leaf = table.detach().requires_grad_()
        out = ssh.embed(leaf, ids.to(DEV), scale=2.0)
        ref.check(out, *ref.embed(table.cpu(), ids, 2.0), "embed")
        back = _randn((3, 17, table.shape[1] * 2), F32, gen)[..., ::2]
        (grad,) = torch.autograd.grad(out, leaf, back.to(DEV))
        ref.check(grad, *ref.embed_grad(back.reshape(51, -1), ids.reshape(-1), table.shape[0], 2.0), "grad")
    row = torch.ones((1, 8), device=DEV).expand(5, 8)  # one row for all tokens
    assert torch.equal(ssh.embed_grad(row, torch.zeros(5, dtype=torch.int64, device=DEV), 2)[0],
                       torch.full((8,), 5.0, device=DEV))


def test_embed_offsets_past_32_bits():
    table = torch.zeros((36, 1 << 26), dtype=BF16, device=DEV)[:, :72]  # rows 128 MiB apart
    value = torch.arange(36 * 72, device=DEV).reshape(36, 72).remainder(251).to(BF16)
    table.copy_(value)
    ids = torch.tensor([35, 0, 33, 34, -1], device=DEV)
    assert torch.equal(ssh.embed(table, ids)[:4], value[ids[:4]])
    del table
    n = (1 << 31) // 256 + 1000
    ids = torch.arange(n, device=DEV, dtype=torch.int32) % 36
    out = ssh.embed(value[:, :64].repeat(1, 4), ids)
    assert torch.equal(out[-2000:], value[:, :64].repeat(1, 4)[ids[-2000:].long()])


# ------------------------------------------------------------------ attention --

def _inputs(q_lens, k_lens, heads, kv_heads, width, dtype, seed, axes=0, mask="full", first=0, std=1.0):
    gen = torch.Generator().manual_seed(seed)
    q_at, k_at = _ends(q_lens, first), _ends(k_lens, first)
    tq, tk = q_at[-1] + first, k_at[-1] + first
    s = dict(q=_randn((tq, heads, width), dtype, gen, std), k=_randn((tk, kv_heads, width), dtype, gen),
             v=_randn((tk, kv_heads, width), dtype, gen), grad=_randn((tq, heads, width), dtype, gen))
    more = dict(causal=mask != "full")
    if mask == "prefix":
        more["prefix"] = torch.tensor([n // 2 for n in k_lens], dtype=torch.int32)
    if axes:
        top = torch.tensor([40, 496, 432])[-axes:]
        more["q_pos"] = (torch.rand((tq, axes), generator=gen) * top).int()
        more["k_pos"] = (torch.rand((tk, axes), generator=gen) * top).int()
        more["slopes"] = 2.0 ** -torch.arange(1, heads + 1).float()
    return s, q_at, k_at, more


def _gpu(t):
    return {n: x.to(DEV) if isinstance(x, torch.Tensor) else x for n, x in t.items()}


def _compare(s, q_at, k_at, more, cap, what):
    scale = s["q"].shape[2] ** -0.5
    want = ref.attend(s["q"], s["k"], s["v"], q_at, k_at, scale, cap=cap, grad=s["grad"],
                      **{n: x for n, x in more.items() if n != "causal"}, causal=more["causal"])
    g, m = _gpu(s), dict(_gpu(more), q_offsets=_at(q_at), k_offsets=_at(k_at), cap=cap)
    print(what, flush=True)
    out, lse = ssh.attend(g["q"], g["k"], g["v"], return_lse=True, **m)
    made = dict(zip(("gq", "gk", "gv"), ssh.attend_grad(g["grad"], g["q"], g["k"], g["v"], out, lse, **m)))
    made.update(out=out)
    assert torch.equal(torch.isinf(lse.cpu()), torch.isinf(want["lse"][0])), what
    there = ~torch.isinf(want["lse"][0])
    ref.check(lse.cpu()[there], want["lse"][0][there], want["lse"][1][there] + 1e-12, what + " lse")
    for n in made:
        ref.check(made[n], *want[n], f"{what} {n}")
    plain = ssh.attend(g["q"], g["k"], g["v"], **m)
    ref.check(plain, *want["out"], what + " out without lse")
    return made


LENGTHS = [([1], [1]), ([31, 0, 33], [31, 7, 33]), ([64, 65, 1], [64, 65, 1]), ([5, 0, 2], [0, 9, 130]),
           ([129, 127], [129, 127]), ([3, 70], [200, 66]), ([0, 0], [0, 3])]


@pytest.mark.parametrize("mask", ["full", "causal", "prefix"])
@pytest.mark.parametrize("heads,kv_heads,width,axes,cap", [
    (2, 2, 32, 0, 0.0), (4, 1, 64, 2, 0.0), (3, 1, 128, 0, 15.0), (8, 2, 48, 3, 20.0), (2, 1, 80, 1, 0.0),
    (2, 1, 8, 0, 0.0), (6, 2, 120, 3, 0.0), (1, 1, 64, 0, 0.5)])
def test_attend(mask, heads, kv_heads, width, axes, cap):
    for i, (q_lens, k_lens) in enumerate(LENGTHS):
        dtype = (BF16, F16)[(i + width // 8) % 2]
        s, q_at, k_at, more = _inputs(q_lens, k_lens, heads, kv_heads, width, dtype, i, axes, mask,
                                      first=(0, 3)[i % 2])
        _compare(s, q_at, k_at, more, cap,
                 f"attend {q_lens} {k_lens} {mask} h {heads}/{kv_heads} w {width} axes {axes} {dtype}")


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("width,axes,cap,mask", [(128, 0, 0.0, "prefix"), (64, 2, 0.0, "full"),
                                                 (128, 2, 0.0, "full"), (64, 0, 30.0, "causal"),
                                                 (32, 3, 20.0, "full"), (128, 0, 30.0, "prefix")])
def test_attend_long(dtype, width, axes, cap, mask):
    """Enough rows for blocks of several wavefronts and many key tiles."""
    s, q_at, k_at, more = _inputs([300, 517], [300, 517], 4, 2, width, dtype, 11, axes, mask)
    _compare(s, q_at, k_at, more, cap, f"attend long w {width} axes {axes} cap {cap} {mask} {dtype}")


@pytest.mark.parametrize("width,axes,cap,mask", [(128, 0, 0.0, "causal"), (64, 2, 0.0, "full"),
                                                 (32, 0, 20.0, "prefix")])
def test_attend_split_queries(width, axes, cap, mask):
    """Few key blocks and many queries: grad_k and grad_v from parts."""
    for lens in ([1100], [1500, 40, 0]):
        s, q_at, k_at, more = _inputs(lens, lens, 4, 2, width, BF16, 12, axes, mask, first=2)
        _compare(s, q_at, k_at, more, cap, f"attend split {lens} w {width} {mask}")


@pytest.mark.parametrize("q_len", [1, 5])
@pytest.mark.parametrize("heads,kv_heads,width,axes,cap", [(16, 4, 128, 0, 0.0), (8, 8, 64, 2, 0.0),
                                                           (4, 1, 80, 0, 20.0), (2, 2, 32, 3, 0.0)])
def test_attend_few_queries_of_long_caches(q_len, heads, kv_heads, width, axes, cap):
    """Keys split into ranges: documents shorter than one of them beside long ones."""
    for k_lens in ([5000], [4100, 3, 0, 2500], [700] * 9):
        for mask in ("full", "prefix"):
            s, q_at, k_at, more = _inputs([q_len] * len(k_lens), k_lens, heads, kv_heads, width, BF16, 5,
                                          axes, mask)
            _compare(s, q_at, k_at, more, cap, f"attend token {k_lens} {mask} w {width}")


def test_attend_concentrated_weights():
    """Softmax rows that are nearly one key: the score gradients cancel."""
    for dtype, mask in ((BF16, "full"), (F16, "causal")):
        s, q_at, k_at, more = _inputs([90, 40], [90, 40], 4, 2, 64, dtype, 8, 2, mask, std=3.0)
        _compare(s, q_at, k_at, more, 20.0, f"concentrated {dtype}")


def test_attend_large_scores_and_first_tiles():
    """Scores far from zero, falling and rising along the keys."""
    gen = torch.Generator().manual_seed(9)
    for sign in (1.0, -1.0):
        s, q_at, k_at, more = _inputs([70], [400], 2, 1, 32, F16, 9)
        s["q"] = _randn((70, 2, 32), F16, gen, 0.1) + 2.0
        s["k"] = s["k"] * 0.25 + (sign * torch.linspace(-8, 8, 400))[:, None, None].half()
        _compare(s, q_at, k_at, more, 0.0, f"large scores {sign}")


def test_attend_rows_that_see_nothing():
    """More queries than keys under a causal mask, and values that are not finite."""
    s, q_at, k_at, more = _inputs([40, 6], [9, 0], 2, 1, 64, BF16, 4, mask="causal")
    made = _compare(s, q_at, k_at, more, 0.0, "nothing seen")
    assert not made["out"][:31].any() and not made["gq"][:31].any()
    g = _gpu(s)
    v = g["v"].clone()
    v[4:9] = math.inf
    v[5] = math.nan
    m = dict(q_offsets=_at(q_at), k_offsets=_at(k_at), causal=True)
    out = ssh.attend(g["q"], g["k"], v, **m)
    assert not out[:31].any() and not out[40:].any()


def test_attend_other_documents_do_not_leak():
    """NaN and infinities in other documents and in rows of no document change nothing."""
    s, q_at, k_at, more = _inputs([30, 33, 50], [45, 33, 80], 4, 2, 64, BF16, 6, 2, "prefix", first=5)
    g = _gpu(s)
    m = dict(_gpu(more), q_offsets=_at(q_at), k_offsets=_at(k_at))
    out, lse = ssh.attend(g["q"], g["k"], g["v"], return_lse=True, **m)
    want = ssh.attend_grad(g["grad"], g["q"], g["k"], g["v"], out, lse, **m)
    bad = {n: t.clone() for n, t in g.items()}
    for n, at in (("q", q_at), ("grad", q_at), ("k", k_at), ("v", k_at)):
        for rows in (slice(0, 5), slice(at[1], at[2]), slice(at[3], None)):
            bad[n][rows] = math.nan
        bad[n][at[1]] = math.inf
    got, got_lse = ssh.attend(bad["q"], bad["k"], bad["v"], return_lse=True, **m)
    grads = ssh.attend_grad(bad["grad"], bad["q"], bad["k"], bad["v"], got, got_lse, **m)
    q_rows = [*range(q_at[0], q_at[1]), *range(q_at[2], q_at[3])]
    k_rows = [*range(k_at[0], k_at[1]), *range(k_at[2], k_at[3])]
    for a, b, rows in ((out, got, q_rows), (want[0], grads[0], q_rows), (want[1], grads[1], k_rows),
                       (want[2], grads[2], k_rows)):
        assert torch.equal(a[rows], b[rows])
    for t, at in ((got, q_at), (grads[0], q_at), (grads[1], k_at), (grads[2], k_at)):
        assert not t[:5].any() and not t[at[3]:].any()


def test_attend_wrong_offsets_stay_inside():
    """Offsets past the tokens or decreasing: some result, no access outside."""
    s, _, _, _ = _inputs([50], [60], 2, 1, 32, F16, 6)
    g = _gpu(s)
    for q_at, k_at in (([0, 90], [-5, 1000]), ([10, 5, 70], [0, 2**31 - 1, 3]), ([-9, -9], [60, 60])):
        m = dict(q_offsets=_at(q_at), k_offsets=_at(k_at), causal=True,
                 prefix=torch.full((len(q_at) - 1,), 2**31 - 1, dtype=torch.int32, device=DEV))
        out, lse = ssh.attend(g["q"], g["k"], g["v"], return_lse=True, **m)
        ssh.attend_grad(g["grad"], g["q"], g["k"], g["v"], out, lse, **m)
        torch.cuda.synchronize()


def test_attend_strides_and_layouts():
    gen = torch.Generator().manual_seed(2)
    tokens, heads, kv_heads, width = 70, 4, 2, 64
    fused = _randn((tokens, heads + 2 * kv_heads, width), BF16, gen).to(DEV)
    q, k, v = fused.split([heads, kv_heads, kv_heads], 1)
    more = dict(causal=True)
    want = ssh.attend(q.contiguous(), k.contiguous(), v.contiguous(), **more)
    assert torch.equal(ssh.attend(q, k, v, **more), want)
    by_head = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v)]  # [heads, tokens, width]
    assert torch.equal(ssh.attend(*by_head, **more), want)
    odd = [torch.nn.functional.pad(t, (3, 2))[..., 3:-2] for t in (q, k, v)]  # not 16-byte aligned
    assert torch.equal(ssh.attend(*odd, **more), want)
    one = k[:, :1].expand(-1, 4, -1)  # a shared key head as a stride of zero
    assert torch.equal(ssh.attend(q, one, one, **more), ssh.attend(q, k[:, :1], k[:, :1], **more))
    out, lse = ssh.attend(q, k, v, return_lse=True, **more)
    g = _randn((tokens, width, heads), BF16, gen).to(DEV).transpose(1, 2)
    a = ssh.attend_grad(g, q, k, v, out, lse, **more)
    b = ssh.attend_grad(g.contiguous(), *by_head, out, lse, **more)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    pos = torch.randint(0, 400, (3, tokens), generator=gen, dtype=torch.int32).to(DEV)
    slopes = torch.full((4,), 0.1, device=DEV)
    a = ssh.attend(q, k, v, slopes=slopes, q_pos=pos.t(), k_pos=pos.t())
    b = ssh.attend(q, k, v, slopes=slopes, q_pos=pos.t().contiguous(), k_pos=pos.t().contiguous())
    assert torch.equal(a, b)


def test_attend_offsets_past_32_bits():
    """One token per 128 MiB of a cache, and a query at its end."""
    gen = torch.Generator().manual_seed(3)
    cache = torch.zeros((36, 1 << 26), dtype=BF16, device=DEV)
    k, v = (_randn((36, 2, 64), BF16, gen) for _ in range(2))
    kk, vv = cache[:, :128].view(36, 2, 64), cache[:, 128:256].view(36, 2, 64)
    kk.copy_(k)
    vv.copy_(v)
    q = _randn((36, 4, 64), BF16, gen)
    at = _at([0, 3, 36])
    want = ref.attend(q, k, v, [0, 3, 36], [0, 3, 36], 0.125, causal=True, grad=q)
    m = dict(q_offsets=at, k_offsets=at, causal=True)
    out, lse = ssh.attend(q.to(DEV), kk, vv, return_lse=True, **m)
    ref.check(out, *want["out"], "far cache")
    made = ssh.attend_grad(q.to(DEV), q.to(DEV), kk, vv, out, lse, **m)
    for n, t in zip(("gq", "gk", "gv"), made):
        ref.check(t, *want[n], "far cache " + n)


def test_attend_autograd_streams_and_repeats():
    s, q_at, k_at, more = _inputs([50, 90], [50, 90], 4, 2, 64, F16, 7, 2, "causal")
    m = dict(_gpu(more), q_offsets=_at(q_at), k_offsets=_at(k_at), cap=20.0)
    g = _gpu(s)
    out, lse = ssh.attend(g["q"], g["k"], g["v"], return_lse=True, **m)
    want = ssh.attend_grad(g["grad"], g["q"], g["k"], g["v"], out, lse, **m)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        leaves = [g[n].clone().requires_grad_() for n in "qkv"]
        again = ssh.attend(*leaves, **m)
        made = torch.autograd.grad(again, leaves, g["grad"])
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(again, out) and all(torch.equal(a, b) for a, b in zip(made, want))


def _replays(step, inputs):
    """A captured step against the eager one, over several replays with eager work between."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        made = step()
    for i in range(4):
        for t in inputs:
            t.copy_(t.flip(0))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in made]
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i


def test_graph_attention():
    s, q_at, k_at, more = _inputs([60, 70, 1], [60, 70, 3000], 4, 2, 64, BF16, 7, 2, "prefix")
    m = dict(_gpu(more), q_offsets=_at(q_at), k_offsets=_at(k_at))
    g = _gpu(s)

    def step():
        out, lse = ssh.attend(g["q"], g["k"], g["v"], return_lse=True, **m)
        return (out, *ssh.attend_grad(g["grad"], g["q"], g["k"], g["v"], out, lse, **m))

    _replays(step, [g["q"], g["k"], g["v"], g["grad"]])


def test_graph_embedding_and_recurrence():
    gen = torch.Generator().manual_seed(2)
    ids = torch.randint(-1, 900, (5000,), generator=gen).to(DEV)
    grad = _randn((5000, 64), F32, gen).to(DEV)
    gate, x = (_randn((5000, 64), F32, gen).to(DEV) for _ in range(2))
    at = _at([0, 4000, 4000, 5000])

    def step():
        y, last, carry = ssh.gated_scan(gate, x, at, return_carry=True)
        return (ssh.embed_grad(grad, ids, 900), ssh.embed(grad, ids), y, last,
                *ssh.gated_scan_grad(grad, gate, x, carry, at))

    _replays(step, [ids, grad, gate, x])


# ----------------------------------------------------------------- recurrence --

SCANS = [[0], [1], [1] * 70, [0, 17, 16, 1, 0, 33], [100, 0, 0, 5], [700], [300, 1000, 64], [9, 0, 2500],
         [2] * 600, [31, 32, 33] * 40]


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("width,dtype", [(1, F32), (33, BF16), (64, F16), (100, F32), (128, BF16),
                                         (256, F16), (260, BF16), (512, F32)])
def test_scan(reverse, width, dtype):
    gen = torch.Generator().manual_seed(width)
    for i, lens in enumerate(SCANS):
        first = (0, 5)[i % 2]
        at = _ends(lens, first)
        t = at[-1] + first
        gate, x, grad = (_randn((t, width), dtype, gen, s) for s in (2.0, 1.0, 1.0))
        gate = (gate.float() + 2.0).to(dtype)
        state = _randn((len(lens), width), F32, gen) if i % 3 else None
        grad_state = _randn((len(lens), width), F32, gen) if i % 3 != 1 else None
        want = ref.scan(gate, x, at, state, reverse, grad, grad_state)
        print(f"scan {lens[:6]}x{len(lens)} width {width} {dtype}", flush=True)
        m = dict(state=None if state is None else state.to(DEV), reverse=reverse)
        y, last, carry = ssh.gated_scan(gate.to(DEV), x.to(DEV), _at(at), return_carry=True, **m)
        y2, last2 = ssh.gated_scan(gate.to(DEV), x.to(DEV), _at(at), **m)
        assert torch.equal(y, y2) and torch.equal(last, last2)
        made = ssh.gated_scan_grad(grad.to(DEV), gate.to(DEV), x.to(DEV), carry, _at(at),
                                   grad_state=None if grad_state is None else grad_state.to(DEV), **m)
        for n, got in zip(("y", "last", "gg", "gx", "gs"), (y, last, *made)):
            ref.check(got, *want[n], f"{n} of {lens[:6]}x{len(lens)} width {width} {dtype}")


@pytest.mark.parametrize("t,width", [(150001, 8), (9000, 130)])
def test_scan_long(t, width):
    """Many chunks, one document and then three; the last documents hold nothing."""
    gen = torch.Generator().manual_seed(t)
    gate, x, grad = (_randn((t, width), F32, gen, s) for s in (1.0, 1.0, 1.0))
    gate += 5.0
    for at, reverse in (([0, t], False), ([0, t // 3, t // 3 + 77, t, t, t], True)):
        print(f"scan t {t} width {width} {at[:3]} reverse {reverse}", flush=True)
        want = ref.scan(gate, x, at, None, reverse, grad)
        y, last, carry = ssh.gated_scan(gate.to(DEV), x.to(DEV), _at(at), reverse=reverse,
                                        return_carry=True)
        made = ssh.gated_scan_grad(grad.to(DEV), gate.to(DEV), x.to(DEV), carry, _at(at),
                                   reverse=reverse)
        for n, got in zip(("y", "last", "gg", "gx", "gs"), (y, last, *made)):
            ref.check(got, *want[n], f"{n} t {t} {at[:3]} {reverse}")


def test_scan_saturated_gates():
    """Gates at 0 and 1 to the last bit, and beyond what exp holds."""
    gate = torch.tensor([[-200.0, -80.0, 0.0, 80.0, 200.0]]).repeat(50, 1)
    x = torch.arange(250.0).reshape(50, 5)
    want = ref.scan(gate, x, [0, 50], torch.ones((1, 5)), grad=torch.ones_like(x))
    y, last, carry = ssh.gated_scan(gate.to(DEV), x.to(DEV), state=torch.ones((1, 5), device=DEV),
                                    return_carry=True)
    made = ssh.gated_scan_grad(torch.ones_like(y), gate.to(DEV), x.to(DEV), carry,
                               state=torch.ones((1, 5), device=DEV))
    for n, got in zip(("y", "last", "gg", "gx", "gs"), (y, last, *made)):
        ref.check(got, *want[n], n)
    assert torch.equal(y[:, 4].cpu(), torch.ones(50)) and torch.equal(y[:, 0].cpu(), x[:, 0])


def test_scan_leaks_nothing_and_wrong_offsets_stay_inside():
    gen = torch.Generator().manual_seed(1)
    gate, x, grad = (_randn((300, 64), F32, gen).to(DEV) for _ in range(3))
    at = _at([10, 100, 220, 290])
    y, last, carry = ssh.gated_scan(gate, x, at, return_carry=True)
    want = ssh.gated_scan_grad(grad, gate, x, carry, at)
    bad = [t.clone() for t in (gate, x, grad)]
    for t in bad:
        t[:10], t[100:220], t[290:] = math.nan, math.inf, math.nan
        t[150] = math.nan
    y2, last2, carry2 = ssh.gated_scan(bad[0], bad[1], at, return_carry=True)
    got = ssh.gated_scan_grad(bad[2], bad[0], bad[1], carry2, at)
    rows = [*range(10, 100), *range(220, 290)]
    assert torch.equal(y[rows], y2[rows]) and torch.equal(last[[0, 2]], last2[[0, 2]])
    for a, b in zip(want[:2], got[:2]):
        assert torch.equal(a[rows], b[rows])
    assert torch.equal(want[2][[0, 2]], got[2][[0, 2]])
    assert not y2[:10].any() and not y2[290:].any() and not got[0][:10].any() and not got[1][290:].any()
    for ends in ([-4, 500], [200, 100, 250], [300, 300], [50, 40, 30, 20]):
        for reverse in (False, True):
            _, _, c = ssh.gated_scan(gate, x, _at(ends), reverse=reverse, return_carry=True)
            ssh.gated_scan_grad(grad, gate, x, c, _at(ends), reverse=reverse)
            torch.cuda.synchronize()


def test_scan_strides_and_autograd():
    gen = torch.Generator().manual_seed(2)
    wide = _randn((90, 300), F32, gen).to(DEV)
    at, state = _at([0, 50, 90]), _randn((2, 100), F32, gen).to(DEV)
    gate, x = wide[:, :100], wide[:, 150:250]
    leaves = [t.detach().requires_grad_() for t in (gate, x, state)]
    y, last = ssh.gated_scan(leaves[0], leaves[1], at, state=leaves[2])
    gy, gl = _randn((100, 90), F32, gen).to(DEV).t(), _randn((2, 100), F32, gen).to(DEV)
    made = torch.autograd.grad((y, last), leaves, (gy, gl))
    want = ref.scan(gate.cpu(), x.cpu(), [0, 50, 90], state.cpu(), grad=gy.cpu(), grad_state=gl.cpu())
    for n, got in zip(("y", "last", "gg", "gx", "gs"), (y, last, *made)):
        ref.check(got, *want[n], n)
    shifted = torch.empty(64 * 40 + 1, device=DEV, dtype=BF16)[1:].view(40, 64)  # 2-byte aligned
    shifted.copy_(_randn((40, 64), BF16, gen))
    assert torch.equal(ssh.gated_scan(shifted, shifted)[0], ssh.gated_scan(shifted.clone(), shifted.clone())[0])


# ------------------------------------------------------------------- refusals --

def test_refusals_on_the_gpu():
    x = torch.zeros((4, 8), device=DEV)
    h = torch.zeros((4, 2, 16), device=DEV, dtype=BF16)
    ids = torch.zeros(4, dtype=torch.int32, device=DEV)
    at = _at([0, 4])
    for call in (
            lambda: ssh.embed(x, ids.float()), lambda: ssh.embed(x[0], ids), lambda: ssh.embed(x.double(), ids),
            lambda: ssh.embed(x, ids.cpu()), lambda: ssh.embed_grad(x, ids[:3], 4),
            lambda: ssh.attend(h, h.half(), h), lambda: ssh.attend(h, h, h[:3]),
            lambda: ssh.attend(h.float(), h, h), lambda: ssh.attend(h[:, :1], h, h),
            lambda: ssh.attend(h[..., :12], h[..., :12], h[..., :12]),
            lambda: ssh.attend(h, h, h, q_offsets=at), lambda: ssh.attend(h, h, h, scale=0.0),
            lambda: ssh.attend(h, h, h, q_offsets=at.long(), k_offsets=at),
            lambda: ssh.attend(h, h, h, q_offsets=at, k_offsets=_at([0, 2, 4])),
            lambda: ssh.attend(h, h, h, cap=-1.0), lambda: ssh.attend(h, h, h, prefix=at),
            lambda: ssh.attend(h, h, h, slopes=x[0, :2]), lambda: ssh.attend(h, h, h, q_pos=ids[:, None]),
            lambda: ssh.attend(h, h, h, slopes=x[0, :2], q_pos=ids[:, None], k_pos=ids[:3, None]),
            lambda: ssh.attend(h, h, h, slopes=x[0, :3], q_pos=ids[:, None], k_pos=ids[:, None]),
            lambda: ssh.attend_grad(h[:3], h, h, h, h, x[:, :2]),
            lambda: ssh.attend_grad(h, h, h, h, h, x),
            lambda: ssh.gated_scan(x, x[:3]), lambda: ssh.gated_scan(x, x.half()),
            lambda: ssh.gated_scan(x, x, at, state=x), lambda: ssh.gated_scan(x, x, at.long()),
            lambda: ssh.gated_scan_grad(x, x, x, x, at), lambda: ssh.gated_scan_grad(x[:2], x, x, x[:1], at)):
        with pytest.raises(ValueError):
            call()


def test_example_learns():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "pillar_tokens.py")
    spec = importlib.util.spec_from_file_location("pillar_tokens", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, answer = example.main(steps=20)
    assert all(math.isfinite(v) for v in losses + answer)
    assert losses[-1] < 0.5 * losses[0], losses


def test_attend_one_visible_key_has_no_score_gradient():
    """Its weight is 1 whatever its score: exactly no gradient of q and k."""
    for q_lens, k_lens, mask in (([5, 3], [1, 1], "full"), ([40, 6], [40, 6], "causal"), ([300], [1], "full")):
        for axes in (0, 2):
            s, q_at, k_at, more = _inputs(q_lens, k_lens, 4, 2, 64, F16, 3, axes, mask)
            made = _compare(s, q_at, k_at, more, 0.0, f"one key {q_lens} {k_lens} {mask}")
            first = [a for a, n in zip(q_at, q_lens)] if mask == "causal" else slice(None)
            assert not made["gq"][first].any()
            if mask == "full":
                assert not made["gk"].any()
