"""Paths of the token operators that only certain sizes and layouts take, and
the promise that nothing outside the tensors is written."""
import itertools
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import sparse_spatial_hashing_amd as ssh  # noqa: E402
import token_reference as ref  # noqa: E402
from sparse_spatial_hashing_amd import tokens  # noqa: E402

DEV = torch.device("cuda:0")
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
E = ref.E
LIB = tokens._lib


def _at(ends):
    return torch.tensor(list(ends), dtype=torch.int32, device=DEV)


def _stream():
    return torch.cuda.current_stream().cuda_stream


# ------------------------------------------------------------------ embedding --

@pytest.mark.parametrize("n,rows,width,dtype", [
    (12000, 214272, 8, F32), (16384, 140000, 3, BF16), (3000, 5000000, 2, F32),  # in LDS: two passes, two, three
    (20000, 300000, 4, F16), (300000, 1 << 24, 1, F32)])                         # through memory: three
def test_embed_grad_sort_passes(n, rows, width, dtype):
    gen = torch.Generator().manual_seed(n)
    ids = (torch.rand(n, generator=gen).double().pow(3.0) * rows).long().clamp(max=rows - 1)
    ids[torch.rand(n, generator=gen) < 0.05] = -1
    ids[:50] = ids[-1] = rows - 1
    g = torch.randn((n, width), generator=gen).to(dtype)
    print(f"embed_grad n {n} rows {rows} width {width}", flush=True)
    for index in (torch.int64, torch.int32):
        got = ssh.embed_grad(g.to(DEV), ids.to(DEV, index), rows, scale=0.5)
        ref.check(got, *ref.embed_grad(g, ids, rows, 0.5), "embed_grad")


# ------------------------------------------------------------------ attention --

@pytest.mark.parametrize("width,heads,axes", [(64, 4, 0), (48, 4, 2), (128, 4, 0), (32, 1, 0)])
def test_attend_far_tokens_in_place(width, heads, axes):
    """Tokens 64 MiB - 16 bytes apart, the farthest that are read where they are: a tile of 64
    spans nearly 2^32 bytes."""
    gen = torch.Generator().manual_seed(width)
    n, ends = 134, [0, 70, 134]
    row = (1 << 25) - 8
    host = {name: torch.randn((n, h, width), generator=gen).to(BF16)
            for name, h in (("q", heads), ("k", 1), ("v", 1), ("g", heads))}
    cache = torch.empty(n * row, dtype=BF16, device=DEV)
    far, start = {}, 0
    for name, t in host.items():
        far[name] = cache.as_strided(t.shape, (row, width, 1), start)
        far[name].copy_(t)
        start += t.shape[1] * width
    more = {}
    if axes:
        pos = torch.randint(0, 60, (n, axes), generator=gen, dtype=torch.int32)
        more = dict(q_pos=pos, k_pos=pos, slopes=2.0 ** -torch.arange(1, heads + 1).float())
    want = ref.attend(host["q"], host["k"], host["v"], ends, ends, width ** -0.5, causal=True,
                      grad=host["g"], **more)
    m = dict({x: t.to(DEV) for x, t in more.items()}, q_offsets=_at(ends), k_offsets=_at(ends), causal=True)
    print(f"far tokens, width {width}", flush=True)
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    out, lse = ssh.attend(far["q"], far["k"], far["v"], return_lse=True, **m)
    made = ssh.attend_grad(far["g"], far["q"], far["k"], far["v"], out, lse, **m)
    assert torch.cuda.max_memory_allocated() - before < 16 << 20
    for name, t in zip(("out", "gq", "gk", "gv"), (out, *made)):
        ref.check(t, *want[name], f"far tokens {name} width {width}")


@pytest.mark.parametrize("q_lens,k_lens,width,axes,cap", [
    ([300, 40], [300, 40], 64, 2, 0.0), ([36] * 9, [36] * 9, 32, 3, 20.0), ([1, 1], [9000, 4000], 128, 0, 0.0),
    ([700], [700], 128, 0, 30.0)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_attend_same_bits_with_and_without_lse(q_lens, k_lens, width, axes, cap, dtype):
    gen = torch.Generator().manual_seed(width)
    q, k, v = (torch.randn((sum(n), h, width), generator=gen).to(DEV, dtype)
               for n, h in ((q_lens, 4), (k_lens, 2), (k_lens, 2)))
    m = dict(q_offsets=_at([0, *itertools.accumulate(q_lens)]), k_offsets=_at([0, *itertools.accumulate(k_lens)]),
             cap=cap)
    if axes:
        m.update(q_pos=torch.randint(0, 99, (sum(q_lens), axes), generator=gen, dtype=torch.int32).to(DEV),
                 k_pos=torch.randint(0, 99, (sum(k_lens), axes), generator=gen, dtype=torch.int32).to(DEV),
                 slopes=torch.tensor([0.5, 0.25, 0.125, 0.0], device=DEV))
    out, _ = ssh.attend(q, k, v, return_lse=True, **m)
    assert torch.equal(ssh.attend(q, k, v, **m), out)


def test_attend_cache_with_room_to_grow():
    """Caches of a fixed room: a document of each cache's keys, one of no queries for the room left.
    What the room holds does not matter, and appending a key is a store and a longer offset."""
    gen = torch.Generator().manual_seed(3)
    caches, room, width = 3, 40, 64
    k, v = (torch.full((caches, room, 2, width), math.nan, dtype=BF16, device=DEV) for _ in range(2))
    lens = [5, 0, 17]
    kept = [[torch.randn((n, 2, width), generator=gen).to(BF16) for n in lens] for _ in range(2)]
    one = torch.arange(caches + 1, dtype=torch.int32, device=DEV)
    q_at = one.repeat_interleave(2)[1:]          # 0 1 1 2 2 3 3: a query, then none, of each cache
    for _ in range(3):
        for c in range(caches):
            for cache, mine in ((k, kept[0]), (v, kept[1])):
                mine[c] = torch.cat([mine[c], torch.randn((1, 2, width), generator=gen).to(BF16)])
                cache[c, lens[c]] = mine[c][-1].to(DEV)
                cache[c, :lens[c]] = mine[c][:-1].to(DEV)
            lens[c] += 1
        starts = torch.arange(caches, device=DEV, dtype=torch.int32) * room
        k_at = torch.cat([torch.stack([starts, starts + _at(lens)], 1).flatten(),
                          torch.full((1,), caches * room, dtype=torch.int32, device=DEV)])
        q = torch.randn((caches, 4, width), generator=gen).to(BF16)
        ends = [0, *itertools.accumulate(lens)]
        want = ref.attend(q, torch.cat(kept[0]), torch.cat(kept[1]), range(caches + 1), ends, 0.125, causal=True)
        out = ssh.attend(q.to(DEV), k.flatten(0, 1), v.flatten(0, 1), q_offsets=q_at, k_offsets=k_at, causal=True)
        ref.check(out, *want["out"], f"caches of {lens}")


# ----------------------------------------------------------------- recurrence --

def _recur(a, b):
    """h[t] = a[t] h[t - 1] + b[t] by doubling the span, in 64 bits."""
    span = 1
    while span < a.shape[0]:
        b = torch.cat([b[:span], b[span:] + a[span:] * b[:-span]])
        a = torch.cat([a[:span], a[span:] * a[:-span]])
        span *= 2
    return b


@pytest.mark.parametrize("reverse", [False, True])
def test_scan_more_chunks_than_are_held(reverse):
    """4.5 M tokens: over 4096 chunks, of which a thread of the prefix reads its share twice."""
    t, width = 4500000, 2
    ends = [3, 8, 1500000, 1500000, 4000123, t - 7]
    docs = len(ends) - 1
    gen = torch.Generator(device=DEV).manual_seed(7)
    gate, x, grad = (torch.randn((t, width), generator=gen, device=DEV) for _ in range(3))
    gate += 4.0
    state, grad_state = (torch.randn((docs, width), generator=gen, device=DEV) for _ in range(2))
    m = dict(state=state, reverse=reverse)
    print(f"scan of {t} tokens, reverse {reverse}", flush=True)
    y, last, carry = ssh.gated_scan(gate, x, _at(ends), return_carry=True, **m)
    made = ssh.gated_scan_grad(grad, gate, x, carry, _at(ends), grad_state=grad_state, **m)
    got = dict(zip(("y", "gg", "gx"), (y, *made[:2])))
    # all in the order of steps
    turn = (lambda z: z.flip(0)) if reverse else (lambda z: z)
    f, z, g = (turn(v).double() for v in (gate, x, grad))
    a, keep = torch.sigmoid(f), torch.sigmoid(-f)
    rel = E * (f.abs() + 8)
    spans = [(t - e, t - b) if reverse else (b, e) for b, e in zip(ends[:-1], ends[1:])]
    some = [(d, b, e) for d, (b, e) in enumerate(spans) if e > b]
    first, final = (torch.tensor([s[i] - (i == 2) for s in some], device=DEV) for i in (1, 2))
    which = torch.tensor([s[0] for s in some], device=DEV)
    inside = torch.zeros((t, 1), dtype=torch.bool, device=DEV)
    for _, b, e in some:
        inside[b:e] = True
    on = a * inside
    on[first] = 0.0                                    # a document starts from its own state
    b = torch.where(inside, keep * z, 0.0)
    b[first] += a[first] * state[which].double()
    size = torch.where(inside, keep * z.abs(), 0.0)
    size[first] += a[first] * state[which].abs().double()
    h, n = _recur(on, b), _recur(on, size)
    off = _recur(on, 2 * (rel + 3 * E) * n)
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    b_off = torch.cat([torch.zeros_like(h[:1]), off[:-1]])
    before[first], b_off[first] = state[which].double(), 0.0
    # from the other end: dh[t] = g[t] + a[t + 1] dh[t + 1]
    def back(values, ends_with):
        w = torch.where(inside, values, 0.0)
        w[final] += ends_with
        after = torch.cat([on[1:], torch.zeros_like(on[:1])])
        return _recur(after.flip(0), w.flip(0)).flip(0)

    dh, dn = back(g, grad_state[which].double()), back(g.abs(), grad_state[which].abs().double())
    d_off = back(2 * (rel + 4 * E) * dn, 0.0)
    k = before - z
    want = {"y": (h, off),
            "gg": (dh * k * a * keep, a * keep * (d_off * k.abs() + dh.abs() * (b_off + 2 * E * k.abs())
                                                  + dh.abs() * k.abs() * (2 * rel + 6 * E))),
            "gx": (dh * keep, (d_off + (rel + 2 * E) * dh.abs()) * keep)}
    tiny = torch.finfo(F32).smallest_normal
    for name, (value, bound) in want.items():
        value, bound = (torch.where(inside, turn_back, 0.0) for turn_back in (value, bound))
        bound = 2 * bound + E * value.abs() + tiny     # two chunked orders of the sum, and the result's rounding
        ref.check(turn(got[name]), value.cpu(), bound.cpu(), f"{name} reverse {reverse}")
    ref.check(last[which], h[final].cpu(), (2 * off[final] + tiny).cpu(), "last state")
    assert torch.equal(last[3 - 1], state[3 - 1])      # the document of no tokens
    ref.check(made[2][which], (dh[first] * a[first]).cpu(),
              (2 * a[first] * d_off[first] + (rel + 2 * E)[first] * 2 * (dh[first] * a[first]).abs() + tiny).cpu(),
              "grad_state")
    assert torch.equal(made[2][3 - 1], grad_state[3 - 1])


# ------------------------------------------------------------ nothing outside --

class Fenced:
    """Tensors each inside a larger buffer of a known byte, which stays around them."""
    ROOM, BYTE = 1 << 16, 0x5A

    def __init__(self):
        self.buffers = []

    def take(self, shape, dtype, fill=None):
        nbytes = math.prod(shape) * dtype.itemsize
        whole = torch.full((2 * self.ROOM + -(-nbytes // 256) * 256,), self.BYTE, dtype=torch.uint8, device=DEV)
        self.buffers.append((whole, nbytes))
        t = whole[self.ROOM:self.ROOM + nbytes]
        t.fill_(0xFF)                                  # NaN in every floating type: nothing may rely on it
        return t.view(dtype).view(shape)

    def check(self):
        torch.cuda.synchronize()
        for whole, nbytes in self.buffers:
            edges = whole[:self.ROOM], whole[self.ROOM + nbytes:]
            assert all(bool((e == self.BYTE).all()) for e in edges), "written outside a tensor"


WRONG = [([0, 90], [-5, 1000]), ([10, 5, 70], [0, 2**31 - 1, 3]), ([-9, -9], [60, 60]),
         ([40, 30, 20, 10], [60, 0, 60, 0]), ([-2**31, 2**31 - 1], [-2**31, 2**31 - 1]), ([0, 50], [0, 60])]


@pytest.mark.parametrize("q_at,k_at", WRONG)
@pytest.mark.parametrize("heads,width,axes,cap,tokens_of", [(2, 32, 0, 0.0, (50, 60)), (4, 64, 2, 0.0, (500, 700)),
                                                            (2, 120, 3, 20.0, (50, 2500))])
def test_attend_writes_nothing_outside(q_at, k_at, heads, width, axes, cap, tokens_of):
    """Offsets past the tokens or decreasing, prefixes out of range, a workspace of NaN."""
    gen = torch.Generator(device=DEV).manual_seed(1)
    (tq, tk), kv = tokens_of, heads // 2
    q, k, v, g = (torch.randn((n, h, width), generator=gen, device=DEV).to(F16)
                  for n, h in ((tq, heads), (tk, kv), (tk, kv), (tq, heads)))
    for prefix in (2**31 - 1, -2**31):
        m = dict(q_offsets=_at(q_at), k_offsets=_at(k_at), scale=0.125, cap=cap, causal=True,
                 prefix=torch.full((len(q_at) - 1,), prefix, dtype=torch.int32, device=DEV),
                 slopes=None, q_pos=None, k_pos=None)
        if axes:
            m.update(slopes=torch.full((heads,), 0.5, device=DEV))
            for name, n in (("q_pos", tq), ("k_pos", tk)):
                m[name] = torch.randint(-2**31, 2**31 - 1, (n, axes), generator=gen, device=DEV, dtype=torch.int32)
        a, kept = tokens._attention(q, k, v, grad=g, **m)
        print(f"fenced attention {q_at} {k_at} w {width} prefix {prefix}", flush=True)
        f = Fenced()
        out, lse = f.take(q.shape, F16), f.take(q.shape[:2], F32)
        nbytes = LIB.tok_attend_workspace_bytes(a)
        ws = f.take((nbytes,), torch.uint8)
        assert LIB.tok_attend(a, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                              ws.data_ptr(), nbytes, _stream()) == 0
        f.check()
        nbytes = LIB.tok_attend_grad_workspace_bytes(a)
        ws, made = f.take((nbytes,), torch.uint8), [f.take(t.shape, F16) for t in (q, k, v)]
        assert LIB.tok_attend_grad(a, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                   g.data_ptr(), *[t.data_ptr() for t in made], ws.data_ptr(), nbytes,
                                   _stream()) == 0
        f.check()
        if (q_at, k_at) == ([0, 50], [0, 60]):         # right offsets: the public calls' bits
            want, want_lse = ssh.attend(q, k, v, return_lse=True, **m)
            assert torch.equal(out, want) and torch.equal(lse, want_lse)
            assert all(torch.equal(x, y) for x, y in zip(made, ssh.attend_grad(g, q, k, v, out, lse, **m)))


@pytest.mark.parametrize("ends", [[-4, 500], [200, 100, 250], [300, 300], [50, 40, 30, 20], [0, 2**31 - 1],
                                  [-2**31, 10, 2**31 - 1, 5], [0, 120, 120, 300], list(range(300, 0, -4))])
@pytest.mark.parametrize("reverse", [0, 1])
@pytest.mark.parametrize("width,dtype,code", [(3, F32, 0), (128, BF16, 1)])
def test_scan_writes_nothing_outside(ends, reverse, width, dtype, code):
    gen = torch.Generator(device=DEV).manual_seed(2)
    t, docs = 300, len(ends) - 1
    gate, x, g = (torch.randn((t, width), generator=gen, device=DEV).to(dtype) for _ in range(3))
    state, gl = (torch.randn((docs, width), generator=gen, device=DEV) for _ in range(2))
    at, f = _at(ends), Fenced()
    y, last = f.take((t, width), dtype), f.take((docs, width), F32)
    carry = f.take((LIB.tok_scan_runs(t), width), F32)
    nbytes = LIB.tok_scan_workspace_bytes(t, width)
    ws = f.take((nbytes,), torch.uint8)
    print(f"fenced scan {ends[:5]} reverse {reverse} w {width}", flush=True)
    assert LIB.tok_scan(gate.data_ptr(), x.data_ptr(), code, t, width, at.data_ptr(), docs, reverse,
                        state.data_ptr(), y.data_ptr(), last.data_ptr(), carry.data_ptr(), ws.data_ptr(), nbytes,
                        _stream()) == 0
    f.check()
    ws, gg, gx, gs = f.take((nbytes,), torch.uint8), f.take((t, width), dtype), f.take((t, width), dtype), \
        f.take((docs, width), F32)
    assert LIB.tok_scan_grad(g.data_ptr(), gate.data_ptr(), x.data_ptr(), carry.data_ptr(), code, t, width,
                             at.data_ptr(), docs, reverse, state.data_ptr(), gl.data_ptr(), gg.data_ptr(),
                             gx.data_ptr(), gs.data_ptr(), ws.data_ptr(), nbytes, _stream()) == 0
    f.check()
    if ends == [0, 120, 120, 300]:
        m = dict(state=state, reverse=bool(reverse))
        want = ssh.gated_scan(gate, x, at, return_carry=True, **m)
        grads = ssh.gated_scan_grad(g, gate, x, carry, at, grad_state=gl, **m)
        for a, b in zip((y, last, carry, gg, gx, gs), (*want, *grads)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("n,rows,width,dtype,code", [(1, 1, 1, F32, 0), (200, 65, 7, BF16, 1), (5000, 77, 33, F16, 2),
                                                     (40000, 900, 8, BF16, 1), (17000, 3, 300, F32, 0)])
def test_embedding_writes_nothing_outside(n, rows, width, dtype, code):
    """Ids of any value, among them those that only 64 bits hold."""
    gen = torch.Generator().manual_seed(n)
    table, g = (torch.randn((m, width), generator=gen).to(DEV, dtype) for m in (rows, n))
    ids = torch.randint(-2, rows + 2, (n,), generator=gen)
    wild = torch.tensor([2**63 - 1, -2**63, 2**32, 2**31, -2**31, rows, -1, 2**32 + 1])
    ids[::3] = wild[torch.randint(0, len(wild), (len(ids[::3]),), generator=gen)]
    for index in (torch.int64, torch.int32):
        i = ids.clamp(-2**31, 2**31 - 1).to(index) if index == torch.int32 else ids
        d, f = i.to(DEV), Fenced()
        print(f"fenced embedding {n} of {rows} by {width} {index}", flush=True)
        out, grad = f.take((n, width), dtype), f.take((rows, width), dtype)
        nbytes = LIB.tok_embed_grad_workspace_bytes(n, rows, width)
        ws = f.take((nbytes,), torch.uint8)
        assert LIB.tok_embed(table.data_ptr(), rows, width, width, code, d.data_ptr(), d.element_size(), n, 1.5,
                             out.data_ptr(), _stream()) == 0
        assert LIB.tok_embed_grad(g.data_ptr(), width, code, d.data_ptr(), d.element_size(), n, rows, width, 1.5,
                                  grad.data_ptr(), ws.data_ptr(), nbytes, _stream()) == 0
        f.check()
        ref.check(out, *ref.embed(table.cpu(), i, 1.5), "embed")
        ref.check(grad, *ref.embed_grad(g.cpu(), i, rows, 1.5), "embed_grad")
