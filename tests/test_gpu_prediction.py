"""Rotary positions, the loss over a table's rows and attention with decay on the
GPU, against their definitions in 64 bits."""
import itertools
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import sparse_spatial_hashing_amd as ssh  # noqa: E402
import prediction_reference as ref  # noqa: E402
from token_reference import check  # noqa: E402

DEV = torch.device("cuda:0")
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _randn(shape, dtype, gen, std=1.0):
    return (torch.randn(shape, generator=gen) * std).to(dtype)


# ------------------------------------------------------------ rotary positions --

@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("width,rotated,axes", [(128, 128, 1), (64, 32, 1), (80, 20, 1), (48, 48, 3), (33, 32, 2),
                                                (2, 2, 1), (6, 6, 3), (100, 60, 3), (7, 2, 1), (128, 128, 2)])
def test_rotate(dtype, interleaved, width, rotated, axes):
    gen = torch.Generator().manual_seed(width + axes)
    freqs = ssh.rotary_frequencies(rotated, axes=axes, device=DEV)
    for tokens, heads, far in ((1, 1, 10), (67, 5, 500), (700, 3, 1 << 20), (0, 2, 1)):
        x = _randn((tokens, heads, width), dtype, gen)
        pos = torch.randint(-far, far, (tokens, axes), generator=gen, dtype=torch.int32)
        print(f"rotate {dtype} {tokens} x {heads} x {width}, {rotated} of {axes} axes, inter {interleaved}", flush=True)
        for inverse in (False, True):
            got = ssh.rotate(x.to(DEV), pos.to(DEV), freqs, interleaved=interleaved, inverse=inverse)
            assert got.dtype == dtype and got.is_contiguous()
            check(got, *ref.rotate(x, pos, freqs.cpu(), interleaved, inverse), "rotate")


def test_rotate_the_farthest_positions():
    gen = torch.Generator().manual_seed(2)
    x = _randn((8, 2, 64), F32, gen)
    pos = torch.tensor([2**31 - 1, -2**31, 2**31 - 2, 2**30 + 1, 0, -1, 1, 123456789], dtype=torch.int32)
    for stretch, context in ((1.0, 0), (8.0, 0), (32.0, 12000)):
        freqs = ssh.rotary_frequencies(64, stretch=stretch, context=context, device=DEV)
        check(ssh.rotate(x.to(DEV), pos.to(DEV), freqs), *ref.rotate(x, pos, freqs.cpu()), "far")


def test_rotate_strides_and_autograd():
    gen = torch.Generator().manual_seed(3)
    wide = _randn((40, 12, 96), BF16, gen)
    pos = torch.randint(0, 400, (40, 4), generator=gen, dtype=torch.int32)
    freqs = ssh.rotary_frequencies(24, axes=2, device=DEV)
    w, p = wide.to(DEV), pos.to(DEV)
    for view in (lambda t: t[:, :8], lambda t: t[:, 2:9, 8:72], lambda t: t[::2, ::3, 4:60], lambda t: t[:, :, 1:38],
                 lambda t: t[:1].expand(40, -1, -1), lambda t: t.transpose(1, 2)[:, :, :12].contiguous()[:, :, ::1],
                 lambda t: t[..., ::2]):
        x = view(wide)
        for q in (lambda t: t[:, :2], lambda t: t[:, 1:4:2]):
            at = q(pos)[:x.shape[0]]
            if x.shape[2] < 24:
                continue
            got = ssh.rotate(view(w), q(p)[:x.shape[0]], freqs)
            check(got, *ref.rotate(x, at, freqs.cpu()), "strided")
    leaf = w[:, :8].detach().requires_grad_()
    out = ssh.rotate(leaf, p[:, :2], freqs, interleaved=True)
    g = _randn((40, 8, 192), BF16, gen)[..., ::2]
    (grad,) = torch.autograd.grad(out, leaf, g.to(DEV))
    check(grad, *ref.rotate(g, pos[:, :2], freqs.cpu(), True, True), "gradient")


# ------------------------------------------------------------------------ loss --

def _loss_case(t, rows, width, dtype, seed, scale=1.0, none=0.1, size=1.0):
    gen = torch.Generator().manual_seed(seed)
    table = _randn((rows, width), dtype, gen, width ** -0.5)
    ids = torch.randint(0, rows, (t,), generator=gen)
    x = (torch.randn((t, width), generator=gen) + 3.0 * table[ids].float()).to(dtype)
    ids[torch.rand(t, generator=gen) < none] = -1
    grad = (torch.rand(t, generator=gen) + 0.5) * size
    return x, table, ids, grad


def _loss_compare(x, table, ids, grad, scale, what):
    print(what, flush=True)
    want = ref.row_loss(x, table, ids, scale, grad)
    args = x.to(DEV), table.to(DEV), ids.to(DEV)
    loss, lse = ssh.row_loss(*args, scale=scale, return_lse=True)
    assert loss.dtype == F32
    made = dict(loss=loss, lse=lse)
    made["gx"], made["gt"] = ssh.row_loss_grad(grad.to(DEV), *args, lse, scale=scale)
    for n in made:
        check(made[n], *want[n], f"{what} {n}")
    return made


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("width", [8, 32, 40, 96, 128, 136, 264, 512])
def test_row_loss(dtype, width):
    for t, rows in ((1, 1), (3, 255), (32, 700), (33, 257), (130, 2049), (700, 512), (129, 31)):
        x, table, ids, grad = _loss_case(t, rows, width, dtype, t + rows + width)
        _loss_compare(x, table, ids, grad, 1.0, f"row_loss {dtype} t {t} rows {rows} width {width}")


@pytest.mark.parametrize("width", [7, 33, 100])
def test_row_loss_odd_widths(width):
    x, table, ids, grad = _loss_case(70, 300, width, BF16, width)
    _loss_compare(x, table, ids, grad, 0.7, f"row_loss width {width}")


# -------------------------------------------------------- attention with decay --

def _ends(lens, first=0):
    return [first] + [first + n for n in itertools.accumulate(lens)]


def _at(ends):
    return torch.tensor(ends, dtype=torch.int32, device=DEV)


def _decay_case(lens, heads, kv_heads, width, dtype, seed, first=0, state=True):
    gen = torch.Generator().manual_seed(seed)
    at = _ends(lens, first)
    t = at[-1] + first
    s = dict(q=_randn((t, heads, width), dtype, gen), k=_randn((t, kv_heads, width), dtype, gen),
             v=_randn((t, kv_heads, width), dtype, gen),
             decay=2.0 ** (-1.0 - 9.0 * torch.arange(heads) / heads), grad=_randn((t, heads, width), dtype, gen))
    s["decay"][-1] = 0.0
    shape = (len(lens), heads, width, width)
    s["state"] = torch.randn(shape, generator=gen) * 3.0 if state else None
    s["grad_state"] = torch.randn(shape, generator=gen) if state else None
    return s, at


def _decay_compare(s, at, what, reverse=False, scale=None):
    print(what, flush=True)
    width = s["q"].shape[2]
    by = width ** -0.5 if scale is None else scale
    want = ref.decay_attend(s["q"], s["k"], s["v"], s["decay"], at, by, s["state"], reverse, s["grad"], s["grad_state"])
    g = {n: x.to(DEV) if x is not None else None for n, x in s.items()}
    more = dict(state=g["state"], scale=scale, reverse=reverse)
    out, last, carry = ssh.decay_attend(g["q"], g["k"], g["v"], g["decay"], _at(at), return_carry=True, **more)
    grads = ssh.decay_attend_grad(g["grad"], g["q"], g["k"], g["v"], g["decay"], carry, _at(at),
                                  grad_state=g["grad_state"], **more)
    made = dict(zip(("gq", "gk", "gv", "gs"), grads), out=out, last=last)
    for n, x in made.items():
        if x is not None:
            value, bound = want[n]
            x = x.cpu().double()
            if made[n].dtype == F16:
                # what the largest number of fp16 may be passed by rounds to it or to infinity
                over = value.abs() + bound > 65504
                assert (x[over] * value[over].sign() > 65504 - bound[over] * 2).all(), f"{what} {n}"
                x, value = torch.where(over, 0, x), torch.where(over, 0, value)
            check(x, value, bound, f"{what} {n}")
    return made


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("width,heads,kv_heads", [(8, 1, 1), (32, 2, 2), (40, 2, 1), (64, 3, 3), (96, 4, 2), (128, 2, 2)])
def test_decay_attend(dtype, reverse, width, heads, kv_heads):
    for lens, first, state in (([1, 1, 1], 0, True), ([3, 0, 70, 33, 1], 0, True), ([200], 2, False),
                               ([31, 32, 64, 5], 3, True), ([0, 0], 1, True)):
        s, at = _decay_case(lens, heads, kv_heads, width, dtype, width + len(lens), first, state)
        _decay_compare(s, at, f"decay {dtype} {lens} first {first} width {width} heads {heads}/{kv_heads}", reverse)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("width,heads,kv_heads,lens", [(128, 2, 1, [700, 1500, 128]), (64, 2, 2, [1, 2100, 129, 0, 256]),
                                                       (32, 4, 2, [3000])])
def test_decay_attend_segments(dtype, width, heads, kv_heads, lens):
    """Documents of several segments, whole ones and ends."""
    s, at = _decay_case(lens, heads, kv_heads, width, dtype, 7, 1)
    _decay_compare(s, at, f"decay segments {dtype} {lens} width {width}")
    _decay_compare(s, at, f"decay segments reverse {dtype} {lens} width {width}", True, 0.3)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("width,heads,kv_heads", [(8, 2, 1), (40, 1, 1), (128, 2, 2)])
def test_decay_steps_next_to_documents(dtype, reverse, width, heads, kv_heads):
    """Sequences that take a step, and some that begin, in one call."""
    for lens, first in (([1] * 40 + [75] + [0, 2, 0, 1, 33], 0), ([0] * 300 + [400], 2), ([129, 1, 130, 2, 1], 1)):
        s, at = _decay_case(lens, heads, kv_heads, width, dtype, 17, first)
        _decay_compare(s, at, f"decay steps and documents {dtype} {len(lens)} width {width}", reverse)


def test_decay_steps_of_many_sequences():
    """More tokens than documents of one segment may have."""
    s, at = _decay_case([1] * 16000 + [900, 2] + [1] * 100, 1, 1, 8, BF16, 19)
    _decay_compare(s, at, "decay steps of many")


def _on_gpu(f, *args, **more):
    """The 64-bit reference with its work on the GPU, its results back on the host."""
    move = lambda x, d: x.to(d) if isinstance(x, torch.Tensor) else x
    with torch.device(DEV):
        made = f(*[move(a, DEV) for a in args], **{n: move(a, DEV) for n, a in more.items()})
    return {n: (v.cpu(), t.cpu()) for n, (v, t) in made.items()}


@pytest.mark.parametrize("rate", [0.0, 1e-6, 0.04, 0.17, 0.174, 0.9, 5.0, 200.0, 1e9, math.inf, -1.0, math.nan])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_decay_any_rate(rate, dtype):
    """From none to all at once; states fall in their registers, or by each chunk."""
    s, at = _decay_case([700, 90], 2, 2, 64, dtype, 11)
    s["decay"][:] = rate
    taken = dict(s, decay=torch.full((2,), 0.0 if not rate > 0 else min(rate, 1000.0)))
    want = ref.decay_attend(taken["q"], taken["k"], taken["v"], taken["decay"], at, 0.125, s["state"], False,
                            s["grad"], s["grad_state"])
    g = {n: x.to(DEV) for n, x in s.items()}
    print(f"decay rate {rate} {dtype}", flush=True)
    out, last, carry = ssh.decay_attend(g["q"], g["k"], g["v"], g["decay"], _at(at), state=g["state"],
                                        return_carry=True)
    made = dict(zip(("gq", "gk", "gv", "gs"),
                    ssh.decay_attend_grad(g["grad"], g["q"], g["k"], g["v"], g["decay"], carry, _at(at),
                                          state=g["state"], grad_state=g["grad_state"])), out=out, last=last)
    for n, x in made.items():
        check(x, *want[n], f"rate {rate} {n}")


def test_decay_long_documents_keep_their_states():
    """Two thousand chunks, with and without a fall; the states are right to float32."""
    for width, heads, lens in ((32, 2, [60000, 4000]), (128, 1, [20000])):
        s, at = _decay_case(lens, heads, heads, width, BF16, 13)
        s["decay"] = torch.tensor([2.0 ** -13, 0.0][:heads])
        g = {n: x.to(DEV) for n, x in s.items()}
        print(f"decay long {lens}", flush=True)
        out, last = ssh.decay_attend(g["q"], g["k"], g["v"], g["decay"], _at(at), state=g["state"])
        for d, n in enumerate(lens):
            for h in range(heads):
                rows = slice(at[d], at[d + 1])
                until = torch.exp(-float(s["decay"][h]) * (n - 1 - torch.arange(n, dtype=torch.float64, device=DEV)))
                k, v = g["k"][rows, h].double(), g["v"][rows, h].double()
                whole = math.exp(-float(s["decay"][h]) * n)
                want = (until[:, None] * k).T @ v + whole * g["state"][d, h].double()
                size = ((until[:, None] * k).square().sum(0)[:, None] * v.square().mean()).sqrt()
                # random roundings of 2^-22 at most of each term, and of float32 sums of n terms
                off = ((last[d, h].double() - want).abs() / (size + want.abs())).max()
                assert off < 2.0 ** -22 + 2.0 ** -24 * math.sqrt(n), (n, h, float(off))
        # the last tokens' outputs, from the states before them
        tail = [at[1] - 40, at[1]]
        head = ssh.decay_attend(g["q"][:tail[0]], g["k"][:tail[0]], g["v"][:tail[0]], g["decay"],
                                state=g["state"][:1])[1]
        want = ref.decay_attend(s["q"][tail[0]:tail[1]], s["k"][tail[0]:tail[1]], s["v"][tail[0]:tail[1]], s["decay"],
                                [0, 40], width ** -0.5, head.cpu())
        check(out[tail[0]:tail[1]], *want["out"], "tail")


@pytest.mark.parametrize("width", [24, 64, 128])
def test_decay_prompt_then_tokens(width):
    """A prompt in chunks, then token by token, is one run; a token's step holds all in float32."""
    s, at = _decay_case([75, 9, 33], 4, 2, width, BF16, width)
    g = {n: x.to(DEV) for n, x in s.items()}
    cut = [n - 6 for n in (75, 9, 33)]
    first = torch.cat([torch.arange(a, a + n) for a, n in zip(at, cut)]).to(DEV)
    print(f"decay prompt then tokens {width}", flush=True)
    out, state = ssh.decay_attend(g["q"][first], g["k"][first], g["v"][first], g["decay"], _at(_ends(cut)),
                                  state=g["state"])
    made = torch.zeros_like(g["q"])
    made[first] = out
    one = _at([0, 1, 2, 3])
    for i in range(6):
        rows = torch.tensor([a + n + i for a, n in zip(at, cut)], device=DEV)
        before = state.clone()
        made[rows], state = ssh.decay_attend(g["q"][rows], g["k"][rows], g["v"][rows], g["decay"], one, state=state)
        step = ref.decay_attend(*(s[n][rows.cpu()] for n in "qkv"), s["decay"], [0, 1, 2, 3], width ** -0.5, before.cpu())
        # in float32: the type's rounding of the result alone
        assert torch.allclose(state.cpu().double(), step["last"][0], rtol=1e-6, atol=1e-5)
        off = (made[rows].cpu().double() - step["out"][0]).abs()
        assert (off <= step["out"][0].abs() * 2.0 ** -8 + step["out"][1] * 2.0 ** -8).all()
    want = ref.decay_attend(s["q"], s["k"], s["v"], s["decay"], at, width ** -0.5, s["state"])
    check(made, *want["out"], "prompt then tokens")
    check(state, *want["last"], "last state")


@pytest.mark.parametrize("size", [1e-6, 1e-3, 40.0])
def test_decay_fp16_sizes(size):
    """States over fp16's largest number, and weights and gradients far under its smallest."""
    s, at = _decay_case([600, 40], 2, 1, 64, F16, 17)
    s["k"], s["v"] = (s["k"].float() * 20).half(), (s["v"].float() * 20).half()  # states of up to 10^5
    s["grad"] = (s["grad"].float() * size).half()
    s["grad_state"] *= size
    s["decay"] = torch.tensor([0.0, 0.01])
    _decay_compare(s, at, f"decay fp16 grad of {size}")
    s["k"], s["v"] = (s["k"].float() * 1e-4).half(), (s["v"].float() * 1e-3).half()
    s["state"] *= 1e-7
    _decay_compare(s, at, f"decay fp16 small keys, grad of {size}")


def test_decay_other_documents_do_not_leak():
    """NaN outside every document and in another one; rows of no document are zeros."""
    for lens in ([40, 300, 7, 200], [1, 1, 1, 1]):
        s, at = _decay_case(lens, 2, 2, 32, BF16, 19, 3)
        for n in "qkv":
            s[n][at[1]:at[2]] = math.nan
            s[n][:3] = math.inf
            s[n][-3:] = math.nan
        s["grad"][at[1]:at[2]] = math.nan
        s["grad"][:3] = math.nan
        g = {n: x.to(DEV) for n, x in s.items()}
        print(f"decay leaks {lens}", flush=True)
        out, last, carry = ssh.decay_attend(g["q"], g["k"], g["v"], g["decay"], _at(at), state=g["state"],
                                            return_carry=True)
        gq, gk, gv, gs = ssh.decay_attend_grad(g["grad"], g["q"], g["k"], g["v"], g["decay"], carry, _at(at),
                                               state=g["state"], grad_state=g["grad_state"])
        for t in (out, gq, gk, gv):
            assert not t[:3].any() and not t[-3:].any()
            assert t[at[0]:at[1]].isfinite().all() and t[at[2]:at[4]].isfinite().all()
        assert last[[0, 2, 3]].isfinite().all() and gs[[0, 2, 3]].isfinite().all() and last[1].isnan().any()


@pytest.mark.parametrize("ends", [[-4, 500], [200, 100, 250], [300, 300], [50, 40, 30, 20], [0, 2**31 - 1],
                                  [-2**31, 10, 2**31 - 1, 5], [0, 120, 120, 300], list(range(300, 0, -2))])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("heads,kv_heads,width", [(2, 1, 32), (3, 3, 96)])
def test_decay_writes_nothing_outside(ends, reverse, heads, kv_heads, width):
    """Wrong offsets, with every output inside a fence and carry and workspace of NaN."""
    from sparse_spatial_hashing_amd import prediction
    from test_gpu_token_paths import Fenced
    lib, stream = prediction._lib, torch.cuda.current_stream().cuda_stream
    gen = torch.Generator(device=DEV).manual_seed(2)
    t, docs = 300, len(ends) - 1
    q, k, v, g = (torch.randn((t, h, width), generator=gen, device=DEV).to(BF16)
                  for h in (heads, kv_heads, kv_heads, heads))
    shape = (docs, heads, width, width)
    state, gl = (torch.randn(shape, generator=gen, device=DEV) for _ in range(2))
    decay = torch.full((heads,), 0.01, device=DEV)
    a, kept, _ = prediction._decay_args(q, k, v, decay, _at(ends), None, reverse, g)
    f = Fenced()
    rows = lib.tok_decay_carry_rows(a)
    out, last, carry = f.take(q.shape, BF16), f.take(shape, F32), f.take((rows, *shape[1:]), F32)
    print(f"fenced decay {ends[:5]} reverse {reverse} w {width}", flush=True)
    ptr = lambda x: x.data_ptr() if x.numel() else None
    assert lib.tok_decay_attend(a, q.data_ptr(), k.data_ptr(), v.data_ptr(), state.data_ptr(), out.data_ptr(),
                                last.data_ptr(), ptr(carry), stream) == 0
    f.check()
    nbytes = lib.tok_decay_grad_workspace_bytes(a)
    ws, made = f.take((nbytes,), torch.uint8), [f.take(x.shape, BF16) for x in (q, k, v)]
    gs = f.take(shape, F32)
    assert lib.tok_decay_attend_grad(a, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), state.data_ptr(),
                                     ptr(carry), gl.data_ptr(), *[x.data_ptr() for x in made], gs.data_ptr(), ptr(ws),
                                     nbytes, stream) == 0
    f.check()
    if ends == [0, 120, 120, 300]:
        m = dict(state=state, reverse=reverse)
        want = ssh.decay_attend(q, k, v, decay, _at(ends), return_carry=True, **m)
        grads = ssh.decay_attend_grad(g, q, k, v, decay, carry, _at(ends), grad_state=gl, **m)
        for x, y in zip((out, last, *made, gs), (*want[:2], *grads)):
            assert torch.equal(x, y)


def test_decay_strides_and_autograd():
    gen = torch.Generator().manual_seed(23)
    wide = _randn((150, 12, 72), BF16, gen)
    w = wide.to(DEV)
    views = ((lambda t: (t[:, :4, :64], t[:, 4:6, :64], t[:, 6:8, 8:])),
             (lambda t: (t[:, ::3, :40], t[:, :1, 16:56], t[:, 7:8, :40])),
             (lambda t: (t[:, :4, 1:41], t[:, 4:6, 1:41].transpose(0, 1).contiguous().transpose(0, 1), t[:, 8:10, 3:43])),
             (lambda t: (t[:, :4, :32], t[:, 4:5, :32].expand(-1, 4, -1), t[:1, 5:9, :32].expand(150, -1, -1))))
    at, decay = [0, 90, 150], torch.tensor([0.0, 0.02, 0.1, 1.0])
    for view in views:
        s = dict(zip("qkv", view(wide)))
        width = s["q"].shape[2]
        s["grad"] = _randn((150, 4, 2 * width), BF16, gen)[..., ::2]
        state = torch.randn((2, 4, width, width), generator=gen)
        want = ref.decay_attend(s["q"], s["k"], s["v"], decay, at, width ** -0.5, state, False, s["grad"],
                                torch.ones_like(state))
        leaves = [x.detach().requires_grad_() for x in view(w)] + [state.to(DEV).requires_grad_()]
        out, last = ssh.decay_attend(*leaves[:3], decay.to(DEV), _at(at), state=leaves[3])
        made = torch.autograd.grad((out, last), leaves, (s["grad"].to(DEV), torch.ones_like(last)))
        for n, x in zip(("out", "last", "gq", "gk", "gv", "gs"), (out, last, *made)):
            check(x, *want[n], n)
    # without a gradient of the states, and from them alone
    leaves = [x.detach().requires_grad_() for x in views[0](w)]
    out, last = ssh.decay_attend(*leaves, decay.to(DEV), _at(at), return_state=False)
    assert last is None
    (out.float().sum()).backward()
    assert all(x.grad.isfinite().all() for x in leaves)
    out, last = ssh.decay_attend(*leaves, decay.to(DEV), _at(at))
    gq, gk = torch.autograd.grad(last.sum(), leaves[:2])
    assert not gq.any() and gk.any()


def test_decay_far_tokens_and_offsets_past_32_bits():
    """Tokens 32 MiB apart: the tensor spans 4 GiB and more."""
    t, width = 150, 64
    far = torch.zeros((t, 1 << 24), dtype=BF16, device=DEV)
    gen = torch.Generator().manual_seed(29)
    s, at = _decay_case([t], 2, 2, width, BF16, 29)
    views = [far[:, i * 256:i * 256 + 2 * width].unflatten(1, (2, width)) for i in range(4)]
    for view, n in zip(views, ("q", "k", "v", "grad")):
        view.copy_(s[n])
    want = ref.decay_attend(s["q"], s["k"], s["v"], s["decay"], at, 0.125, None, False, s["grad"])
    out, _, carry = ssh.decay_attend(*views[:3], s["decay"].to(DEV), return_carry=True)
    grads = ssh.decay_attend_grad(views[3], *views[:3], s["decay"].to(DEV), carry)
    for n, x in zip(("out", "gq", "gk", "gv"), (out, *grads)):
        check(x, *want[n], "far " + n)


# ------------------------------------------------------------- the loss's edges --

@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("t,rows,width", [(300, 70001, 64), (4, 214272, 128), (40, 30000, 1000), (2500, 9000, 136),
                                          (33, 50000, 32)])
def test_row_loss_long(dtype, t, rows, width):
    """Rows split between blocks, and partial sums of the gradients."""
    x, table, ids, grad = _loss_case(t, rows, width, dtype, t)
    print(f"row_loss long {t} {rows} {width} {dtype}", flush=True)
    want = _on_gpu(ref.row_loss, x, table, ids, 1.5, grad=grad)
    args = x.to(DEV), table.to(DEV), ids.to(DEV)
    loss, lse = ssh.row_loss(*args, scale=1.5, return_lse=True)
    gx, gt = ssh.row_loss_grad(grad.to(DEV), *args, lse, scale=1.5)
    for n, v in (("loss", loss), ("lse", lse), ("gx", gx), ("gt", gt)):
        check(v, *want[n], n)
    again = ssh.row_loss_grad(grad.to(DEV), *args, lse, scale=1.5)
    assert torch.equal(loss, ssh.row_loss(*args, scale=1.5)) and all(torch.equal(a, b) for a, b in zip((gx, gt), again))


@pytest.mark.parametrize("width", [48, 200])
def test_row_loss_rows_far_apart(width):
    """Rows and tokens 8 MiB apart: past 2^32 bytes, and the widest strides that are read in place."""
    t, rows, stride = 290, 700, 2**22 - 8
    x, table, ids, grad = _loss_case(t, rows, width, BF16, 31)
    far = torch.empty(rows * stride, dtype=BF16, device=DEV).view(rows, stride)
    at, from_table = far[:t, 1000:1000 + width], far[:, :width]
    at.copy_(x)
    from_table.copy_(table)
    print(f"row_loss far apart {width}", flush=True)
    want = ref.row_loss(x, table, ids, 1.0, grad)
    loss, lse = ssh.row_loss(at, from_table, ids.to(DEV), return_lse=True)
    gx, gt = ssh.row_loss_grad(grad.to(DEV), at, from_table, ids.to(DEV), lse)
    for n, v in (("loss", loss), ("lse", lse), ("gx", gx), ("gt", gt)):
        check(v, *want[n], n)


def test_row_loss_millions_of_tokens():
    """dZ of 256 rows past 2^32 bytes; every token stands for one of a few hundred."""
    t, rows, width, few = 8400000, 300, 8, 400
    x, table, ids, grad = _loss_case(few, rows, width, BF16, 37)
    which = torch.randint(0, few, (t,), generator=torch.Generator().manual_seed(2))
    print("row_loss millions", flush=True)
    want = ref.row_loss(x, table, ids, 1.0, grad)
    d = which.to(DEV)
    args = x.to(DEV)[d], table.to(DEV), ids.to(DEV)[d]
    loss, lse = ssh.row_loss(*args, return_lse=True)
    gx, gt = ssh.row_loss_grad(grad.to(DEV)[d], *args, lse)
    for n, v in (("loss", loss), ("lse", lse), ("gx", gx)):
        value, bound = want[n]
        for b in (0, t // 2, t - 5000):
            at = which[b:b + 5000]
            check(v[b:b + 5000], value[at], bound[at], n)
    # the table's gradient, token by token of the few: how often each came
    total, bound = torch.zeros(gt.shape, dtype=torch.float64), torch.zeros(gt.shape, dtype=torch.float64)
    for i, n in enumerate(torch.bincount(which, minlength=few).tolist()):
        value, tol = ref.row_loss(x[i:i + 1], table, ids[i:i + 1], 1.0, grad[i:i + 1])["gt"]
        total += n * value
        bound += n * (tol + value.abs() * 2.0 ** -8)  # of one token dZ is in two parts there, in one here
    # t additions of at most the terms' absolute sum, whose 2^-8 is in the bound, at 2^-24 for
    # each of the at most t / 32 + 2 that a sum passes
    check(gt, total, bound * (1 + (t / 32 + 2) * 2.0 ** -24 / 2.0 ** -8) + total.abs() * 2.0 ** -8, "gt")


@pytest.mark.parametrize("width", [32, 256])
def test_row_loss_several_pieces(width):
    """More rows than a piece of dZ holds (256 MB of 20,000 tokens: 6,656 rows), the last one short."""
    t, rows = 20000, 14000
    x, table, ids, grad = _loss_case(t, rows, width, BF16, 3)
    print(f"row_loss pieces {width}", flush=True)
    args = x.to(DEV), table.to(DEV), ids.to(DEV)
    loss, lse = ssh.row_loss(*args, return_lse=True)
    gx, gt = ssh.row_loss_grad(grad.to(DEV), *args, lse)
    some = torch.randperm(t, generator=torch.Generator().manual_seed(1))[:300]
    want = _on_gpu(ref.row_loss, x[some], table, ids[some], 1.0, grad=grad[some])
    for n, v in (("loss", loss), ("lse", lse), ("gx", gx)):
        check(v.cpu()[some], *want[n], n)
    total, bound = torch.zeros(gt.shape, dtype=torch.float64), torch.zeros(gt.shape, dtype=torch.float64)
    for b in range(0, t, 2000):
        part = _on_gpu(ref.row_loss, x[b:b + 2000], table, ids[b:b + 2000], 1.0, grad=grad[b:b + 2000])["gt"]
        total += part[0]
        bound += part[1]
    # a sum of t terms instead of 2,000: their roundings, of terms of at most the parts' bounds / 2^-9
    check(gt, total, bound * (1 + t * 2.0 ** -24 / 2.0 ** -9) + total.abs() * 2.0 ** -8, "gt")


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_row_loss_large_logits(dtype):
    """Logits of hundreds either way, rising along the rows and falling: the maximum lags and is caught up with."""
    gen = torch.Generator().manual_seed(5)
    for width, order in ((32, 1), (64, -1), (160, 1)):
        x = _randn((140, width), dtype, gen).abs() + 0.5
        table = (torch.linspace(-3 * order, 3 * order, 3000)[:, None] * torch.rand((3000, width), generator=gen)).to(dtype)
        ids, grad = torch.randint(0, 3000, (140,), generator=gen), torch.rand(140, generator=gen)
        _loss_compare(x.to(dtype), table, ids, grad, 4.0, f"large logits {width} {order} {dtype}")
    # one row takes all; all rows alike
    x, table = torch.ones((5, 64), dtype=dtype), torch.zeros((700, 64), dtype=dtype)
    _loss_compare(x, table, torch.arange(5), torch.ones(5), 1.0, "all alike")
    table[69] = 8.0
    _loss_compare(x, table, torch.tensor([69, 69, 0, 1, 699]), torch.ones(5), 1.0, "one row")


def test_row_loss_tokens_without_a_row():
    """Nothing of them enters a result, whatever they hold; ids past either end, in both types."""
    for width in (32, 128, 200):
        x, table, ids, grad = _loss_case(90, 400, width, BF16, 7, none=0.3)
        gone = ids < 0
        want = ref.row_loss(x, table, ids, 1.0, grad)
        x[gone] = math.nan
        x[gone.nonzero()[0]] = math.inf
        grad[gone] = math.nan
        ids[gone.nonzero()[1:]] = 400
        for index, far in ((torch.int32, 2**31 - 1), (torch.int64, 2**40 + 3)):
            i = ids.to(index)
            i[gone.nonzero()[-1]] = far
            args = x.to(DEV), table.to(DEV), i.to(DEV)
            loss, lse = ssh.row_loss(*args, return_lse=True)
            gx, gt = ssh.row_loss_grad(grad.to(DEV), *args, lse)
            for n, v in (("loss", loss), ("lse", lse), ("gx", gx), ("gt", gt)):
                check(v, *want[n], f"without a row {n}")
            assert not loss[gone.to(DEV)].any() and not gx[gone.to(DEV)].any()
    args = x.to(DEV), table.to(DEV), torch.full((90,), -1, device=DEV)
    assert not ssh.row_loss(*args).any()
    assert not any(v.any() for v in ssh.row_loss_grad(torch.ones(90, device=DEV), *args, torch.zeros(90, device=DEV)))


def test_row_loss_of_no_tokens_and_shapes():
    table = torch.ones((300, 40), dtype=F16, device=DEV)
    for shape in ((0,), (3, 0), ()):
        ids = torch.zeros(shape, dtype=torch.int32, device=DEV)
        x = torch.ones((*shape, 40), dtype=F16, device=DEV)
        loss, lse = ssh.row_loss(x, table, ids, return_lse=True)
        assert loss.shape == shape and lse.shape == shape
        gx, gt = ssh.row_loss_grad(torch.ones(shape, device=DEV), x, table, ids, lse)
        assert gx.shape == x.shape and gt.shape == table.shape and (ids.numel() or not gt.any())
    x, table, ids, grad = _loss_case(24, 90, 48, BF16, 9)
    flat = ssh.row_loss(x.to(DEV), table.to(DEV), ids.to(DEV))
    assert torch.equal(ssh.row_loss(x.view(4, 6, 48).to(DEV), table.to(DEV), ids.view(4, 6).to(DEV)), flat.view(4, 6))


def test_row_loss_bad_numbers_stay_in_their_token():
    x, table, ids, grad = _loss_case(200, 900, 64, BF16, 11, none=0.0)
    good = ssh.row_loss(x.to(DEV), table.to(DEV), ids.to(DEV))
    x[17, 3], x[150, 0] = math.nan, math.inf
    args = x.to(DEV), table.to(DEV), ids.to(DEV)
    loss, lse = ssh.row_loss(*args, return_lse=True)
    rest = torch.ones(200, dtype=torch.bool, device=DEV)
    rest[[17, 150]] = False
    assert torch.equal(loss[rest], good[rest]) and not loss[~rest].isfinite().any()
    gx, gt = ssh.row_loss_grad(grad.to(DEV), *args, lse)
    assert gx[rest].isfinite().all() and not gx[~rest].isfinite().all() and not gt.isfinite().all()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("size", [1e-9, 1e-5, 1.0, 1e4])
def test_row_loss_gradients_of_any_size(dtype, size):
    """In fp16 the rounded products carry a power of two; gradients under its smallest normal
    number are steps of its smallest."""
    x, table, ids, grad = _loss_case(150, 700, 64, dtype, 13, size=size)
    tiny = torch.finfo(dtype).smallest_normal
    want = ref.row_loss(x, table, ids, 1.0, grad)
    args = x.to(DEV), table.to(DEV), ids.to(DEV)
    _, lse = ssh.row_loss(*args, return_lse=True)
    for n, v in zip(("gx", "gt"), ssh.row_loss_grad(grad.to(DEV), *args, lse)):
        value, bound = want[n]
        bound = (bound - tiny).clamp(min=0) + tiny * torch.finfo(dtype).eps / 2
        over = value.abs() > 65500 if dtype == F16 else torch.zeros_like(value, dtype=torch.bool)
        check(torch.where(over, 0, v.cpu().double()), torch.where(over, 0, value), bound, f"{n} of {size}")


def test_row_loss_strides_and_autograd():
    gen = torch.Generator().manual_seed(15)
    wide_x, wide_t = _randn((200, 100), BF16, gen), _randn((500, 100), BF16, gen)
    ids, grad = torch.randint(-1, 60, (100,), generator=gen), torch.rand(100, generator=gen)
    for view in (lambda t: t[::2, :64], lambda t: t[::2, 8:72], lambda t: t[:100, 1:41], lambda t: t[:100, ::2],
                 lambda t: t[:100, :96], lambda t: t[:1, :64].expand(100, -1), lambda t: t.t()[:100, :64]):
        x, table = view(wide_x), view(wide_t)
        want = ref.row_loss(x, table, ids, 0.5, grad)
        leaves = [view(wide_x.to(DEV)).detach().requires_grad_(), view(wide_t.to(DEV)).detach().requires_grad_()]
        loss, lse = ssh.row_loss(*leaves, ids.to(DEV), scale=0.5, return_lse=True)
        assert not lse.requires_grad
        made = torch.autograd.grad(loss, leaves, grad.to(DEV))
        for n, v in zip(("loss", "lse", "gx", "gt"), (loss, lse, *made)):
            check(v, *want[n], n)
    leaf = wide_x[:, :64].to(DEV).requires_grad_()
    ssh.row_loss(leaf[:60], leaf[:80], ids[:60].to(DEV)).mean().backward()  # both from one tensor
    assert leaf.grad[:60].any() and leaf.grad[60:80].any() and not leaf.grad[80:].any()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("t,rows,width", [(0, 9, 16), (7, 40, 24), (300, 700, 100), (500, 9000, 136)])
def test_row_loss_one_gradient(dtype, t, rows, width):
    """The same as of both, where the other is of a constant."""
    gen = torch.Generator().manual_seed(t)
    x, table = _randn((t, width), dtype, gen).to(DEV), _randn((rows, width), dtype, gen).to(DEV)
    ids, grad = torch.randint(0, rows, (t,), generator=gen).to(DEV), torch.rand(t, generator=gen).to(DEV)
    _, lse = ssh.row_loss(x, table, ids, return_lse=True)
    both = ssh.row_loss_grad(grad, x, table, ids, lse)
    for n in (0, 1):
        leaves = [x.clone(), table.clone()]
        leaves[n].requires_grad_()
        print(f"row loss, one gradient {dtype} {t} {rows} {width} {n}", flush=True)
        ssh.row_loss(*leaves, ids).backward(grad)
        assert torch.equal(leaves[n].grad, both[n]) and leaves[1 - n].grad is None


def test_row_loss_writes_nothing_outside():
    from sparse_spatial_hashing_amd import prediction
    from test_gpu_token_paths import Fenced
    lib, stream = prediction._lib, torch.cuda.current_stream().cuda_stream
    gen = torch.Generator(device=DEV).manual_seed(2)
    for t, rows, width, dtype, code in ((1, 1, 8, BF16, 1), (33, 257, 96, F16, 2), (129, 1025, 40, BF16, 1),
                                        (20, 777, 264, F16, 2), (300, 513, 520, BF16, 1), (700, 90, 128, F16, 2)):
        x, table = (torch.randn((n, width), generator=gen, device=DEV).to(dtype) for n in (t, rows))
        ids = torch.randint(-3, rows + 3, (t,), generator=gen, device=DEV)
        grad = torch.rand(t, generator=gen, device=DEV)
        f = Fenced()
        loss, lse = f.take((t,), F32), f.take((t,), F32)
        gx, gt = f.take((t, width), dtype), f.take((rows, width), dtype)
        print(f"fenced row_loss {t} {rows} {width}", flush=True)
        common = (x.data_ptr(), width, table.data_ptr(), width, code, t, rows, width, ids.data_ptr(), 8)
        nbytes = lib.tok_row_loss_workspace_bytes(t, rows, width)
        ws = f.take((nbytes,), torch.uint8)
        assert lib.tok_row_loss(*common, 0.5, loss.data_ptr(), lse.data_ptr(), ws.data_ptr(), nbytes, stream) == 0
        f.check()
        nbytes = lib.tok_row_loss_grad_workspace_bytes(t, rows, width)
        ws = f.take((nbytes,), torch.uint8)
        assert lib.tok_row_loss_grad(grad.data_ptr(), *common, lse.data_ptr(), 0.5, gx.data_ptr(), gt.data_ptr(),
                                     ws.data_ptr(), nbytes, stream) == 0
        f.check()
        want, want_lse = ssh.row_loss(x, table, ids, scale=0.5, return_lse=True)
        assert torch.equal(loss, want) and torch.equal(lse, want_lse)
        for a, b in zip((gx, gt), ssh.row_loss_grad(grad, x, table, ids, lse, scale=0.5)):
            assert torch.equal(a, b)


# ------------------------------------------------------------------- together --

def _step_inputs(seed):
    gen = torch.Generator().manual_seed(seed)
    heads, width, cells, lens = 4, 32, 700, [90, 1, 200]
    at = _ends(lens)
    model = heads * width
    s = dict(table=_randn((cells, model), BF16, gen, model ** -0.5), ids=torch.randint(0, cells, (at[-1],), generator=gen),
             mix=[_randn((model, model), BF16, gen, model ** -0.5) for _ in range(3)],
             pos=torch.randint(0, 400, (at[-1], 2), generator=gen, dtype=torch.int32),
             decay=torch.tensor([0.0, 0.01, 0.1, 0.5]))
    s["next"] = s["ids"].roll(-1)
    s["next"][[a - 1 for a in at[1:]]] = -1
    return s, at, heads, width


def _step(s, at, heads, width, freqs):
    """Cells in, the next cells' loss out: all operators, the table at both ends."""
    x = ssh.embed(s["table"], s["ids"], scale=4.0)
    q, k, v = ((x @ m).unflatten(1, (heads, width)) for m in s["mix"])
    q, k = ssh.rotate(q, s["pos"], freqs), ssh.rotate(k, s["pos"], freqs)
    near = ssh.attend(q, k, v, q_offsets=at, k_offsets=at, causal=True)
    far, _ = ssh.decay_attend(q, k, v, s["decay"], at, return_state=False)
    x = x + near.flatten(1) + 0.25 * far.flatten(1)
    return ssh.row_loss(x, s["table"], s["next"], scale=2.0)


def test_a_training_step_of_all_operators():
    """Its loss and the table's gradient, against the same step from definitions in 64 bits."""
    s, at, heads, width = _step_inputs(1)
    freqs = ssh.rotary_frequencies(width, axes=2, device=DEV)
    g = {n: [m.to(DEV).requires_grad_() for m in x] if n == "mix" else x.to(DEV) for n, x in s.items()}
    g["table"].requires_grad_()
    loss = _step(g, _at(at), heads, width, freqs)
    (loss.sum() / 288).backward()

    table = s["table"].double().requires_grad_()
    mix = [m.double().requires_grad_() for m in s["mix"]]
    x = table[s["ids"]] * 4.0
    q, k, v = ((x @ m).unflatten(1, (heads, width)) for m in mix)
    turn = s["pos"].double()[:, :, None] * freqs.cpu()
    turn = torch.polar(torch.ones_like(turn), turn)[:, None]
    q, k = ((torch.complex(*t.unflatten(2, (2, 2, width // 4)).unbind(3)) * turn) for t in (q, k))
    q, k = (torch.stack([t.real, t.imag], 3).flatten(2) for t in (q, k))
    seen = []
    for b, e in zip(at[:-1], at[1:]):
        z = torch.einsum("ihc,jhc->hij", q[b:e], k[b:e]) * width ** -0.5
        i = torch.arange(e - b)
        behind = i[:, None] - i[None]
        p = torch.softmax(z.masked_fill(behind < 0, -math.inf), 2)
        w = torch.where(behind >= 0, torch.exp(-s["decay"].double()[:, None, None] * behind.clamp(min=0)), 0.0) * z
        seen.append(torch.einsum("hij,jhc->ihc", p + 0.25 * w, v[b:e]).flatten(1))
    y = (x + torch.cat(seen)) @ table.T * 2.0
    has = s["next"] >= 0
    want = torch.logsumexp(y, 1) - y.gather(1, s["next"].clamp(min=0)[:, None])[:, 0]
    want = torch.where(has, want, 0.0)
    (want.sum() / 288).backward()
    off = lambda a, b: float((a.detach().cpu().double() - b.detach()).norm() / b.detach().norm())
    # some ten roundings to bf16 (2^-9 each, of random sign) lie between the cells and the loss
    assert off(loss, want) < 2.0 ** -6, off(loss, want)
    assert off(g["table"].grad, table.grad) < 2.0 ** -5
    for a, b in zip(g["mix"], mix):
        assert off(a.grad, b.grad) < 2.0 ** -5


def test_streams_and_repeats():
    s, at, heads, width = _step_inputs(2)
    freqs = ssh.rotary_frequencies(width, axes=2, device=DEV)
    g = {n: [m.to(DEV) for m in x] if n == "mix" else x.to(DEV) for n, x in s.items()}
    offsets = _at(at)

    def run():
        leaf = g["table"].detach().clone().requires_grad_()
        loss = _step(dict(g, table=leaf), offsets, heads, width, freqs)
        (grad,) = torch.autograd.grad(loss.sum(), leaf)
        return loss.detach(), grad

    want = run()
    sides = [torch.cuda.Stream() for _ in range(3)]
    made = []
    for side in sides:
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            made.append(run())
    for side in sides:
        torch.cuda.current_stream().wait_stream(side)
    for got in made:
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_graphs():
    from test_gpu_tokens import _replays
    for dtype, lens in ((BF16, [300, 500]), (F16, [1] * 40), (F16, [20, 30] * 40)):
        s, at = _decay_case(lens, 4, 2, 32, dtype, 31)
        g, offsets = {n: x.to(DEV) for n, x in s.items()}, _at(at)
        x, table, ids, grad = (t.to(DEV) for t in _loss_case(120, 900, 40, dtype, 33))
        freqs = ssh.rotary_frequencies(32, device=DEV)
        pos = torch.arange(at[-1], dtype=torch.int32, device=DEV)

        def step():
            q = ssh.rotate(g["q"], pos, freqs)
            out, last, carry = ssh.decay_attend(q, g["k"], g["v"], g["decay"], offsets, state=g["state"],
                                                return_carry=True)
            grads = ssh.decay_attend_grad(g["grad"], q, g["k"], g["v"], g["decay"], carry, offsets, state=g["state"],
                                          grad_state=g["grad_state"])
            loss, lse = ssh.row_loss(x, table, ids, return_lse=True)
            return (q, out, last, *grads, loss, *ssh.row_loss_grad(grad, x, table, ids, lse))

        _replays(step, [g["q"], g["k"], g["v"], g["grad"], g["state"], x, table, grad])


def test_rotate_offsets_past_32_bits_and_many_tokens():
    freqs = ssh.rotary_frequencies(64, device=DEV)
    far = torch.zeros((36, 1 << 26), dtype=BF16, device=DEV)[:, :128].unflatten(1, (2, 64))  # 128 MiB apart
    gen = torch.Generator().manual_seed(35)
    x = _randn((36, 2, 64), BF16, gen)
    far.copy_(x)
    pos = torch.arange(36, dtype=torch.int32)
    check(ssh.rotate(far, pos.to(DEV), freqs), *ref.rotate(x, pos, freqs.cpu()), "far")
    del far
    n = (1 << 31) // 64 + 1000
    x = torch.ones((1, 1, 64), dtype=BF16, device=DEV).expand(n, 1, 64)
    pos = (torch.arange(n, device=DEV) % 1000).int()
    out = ssh.rotate(x, pos, freqs)
    assert torch.equal(out[-3000:], out[(n - 3000) % 1000:][:3000])
    # more blocks than one launch holds: a thread for each pair
    n = 35_000_000
    odd = torch.ones((1, 1, 62), dtype=torch.float16, device=DEV)[:, :, :61].expand(n, 1, 61)
    pos = (torch.arange(n, device=DEV) % 1000).int()
    out = ssh.rotate(odd, pos, freqs[:, :30].contiguous())
    assert torch.equal(out[-3000:], out[(n - 3000) % 1000:][:3000])


def test_refusals_on_the_gpu():
    h = torch.zeros((6, 4, 16), dtype=BF16, device=DEV)
    pos, freqs = torch.zeros(6, dtype=torch.int32, device=DEV), ssh.rotary_frequencies(16, device=DEV)
    rate, at = torch.zeros(4, device=DEV), _at([0, 6])
    x, table, ids = h[:, 0], torch.zeros((9, 16), dtype=BF16, device=DEV), torch.zeros(6, dtype=torch.int64, device=DEV)
    lse, state = torch.zeros(6, device=DEV), torch.zeros((1, 4, 16, 16), device=DEV)
    carry = torch.zeros((0, 4, 16, 16), device=DEV)
    for call in (lambda: ssh.rotate(h[0], pos, freqs), lambda: ssh.rotate(h.double(), pos, freqs),
                 lambda: ssh.rotate(h, pos[:5], freqs), lambda: ssh.rotate(h, pos.long(), freqs),
                 lambda: ssh.rotate(h, pos, freqs.float()), lambda: ssh.rotate(h, pos, freqs.repeat(2, 1)),
                 lambda: ssh.rotate(h, pos, ssh.rotary_frequencies(18, device=DEV)),
                 lambda: ssh.rotate(h, pos.cpu(), freqs), lambda: ssh.rotate(h, pos[:, None].expand(6, 4), freqs),
                 lambda: ssh.decay_attend(h, h[:5], h[:5], rate), lambda: ssh.decay_attend(h, h, h[:, :2], rate),
                 lambda: ssh.decay_attend(h, h[:, :3], h[:, :3], rate), lambda: ssh.decay_attend(h, h, h, rate[:3]),
                 lambda: ssh.decay_attend(h, h, h, rate.double()), lambda: ssh.decay_attend(h, h.half(), h, rate),
                 lambda: ssh.decay_attend(h.float(), h.float(), h.float(), rate),
                 lambda: ssh.decay_attend(h, h, h, rate, at.long()), lambda: ssh.decay_attend(h, h, h, rate, at, scale=0.0),
                 lambda: ssh.decay_attend(h, h, h, rate, at, state=state[:, :3]),
                 lambda: ssh.decay_attend(h, h, h, rate, at, state=state.half()),
                 lambda: ssh.decay_attend(h[:, :, :4], h[:, :, :4], h[:, :, :4], rate),
                 lambda: ssh.decay_attend(*[h.repeat(1, 1, 9)] * 3, rate),
                 lambda: ssh.decay_attend_grad(h[:5], h, h, h, rate, carry),
                 lambda: ssh.decay_attend_grad(h, h, h, h, rate, state),
                 lambda: ssh.decay_attend_grad(h, h, h, h, rate, None),
                 lambda: ssh.decay_attend_grad(h, h, h, h, rate, carry, grad_state=state[..., :8]),
                 lambda: ssh.row_loss(x.float(), table.float(), ids), lambda: ssh.row_loss(x, table.half(), ids),
                 lambda: ssh.row_loss(x, table[:, :8], ids), lambda: ssh.row_loss(x, table[:0], ids),
                 lambda: ssh.row_loss(x, table[0], ids), lambda: ssh.row_loss(x[:5], table, ids),
                 lambda: ssh.row_loss(x, table, ids.float()), lambda: ssh.row_loss(x, table, ids, scale=-1.0),
                 lambda: ssh.row_loss(x, table, ids.cpu()),
                 lambda: ssh.row_loss_grad(lse[:5], x, table, ids, lse), lambda: ssh.row_loss_grad(lse, x, table, ids, lse.half()),
                 lambda: ssh.row_loss_grad(lse.half(), x, table, ids, lse)):
        with pytest.raises(ValueError):
            call()


def test_example_of_the_next_pillar():
    """It runs, every parameter has a gradient, and the loss's is that of its definition."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "pillar_tokens.py")
    spec = importlib.util.spec_from_file_location("pillar_tokens_next", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, answer, model = example.main_next(steps=4)
    assert len(losses) == 4 and len(answer) == 3 and all(math.isfinite(v) for v in losses + answer)
    for name, p in model.named_parameters():
        assert p.grad.isfinite().all() and p.grad.any(), name
    (means, ids, places, offsets), _, _ = example.frames_of(DEV, counts=(300,))
    x = model(means, ids, places, offsets)[0].detach().requires_grad_()
    following = ids.roll(-1)
    following[-1] = -1
    loss = model.loss(x, following)
    grad = torch.autograd.grad(loss.sum(), x)[0]
    table = model.cells.detach().bfloat16()
    want = _on_gpu(ref.row_loss, x.detach(), table, following, 1.0, grad=torch.ones(ids.shape[0]))
    check(loss, *want["loss"], "loss")
    check(grad, *want["gx"], "gradient")
