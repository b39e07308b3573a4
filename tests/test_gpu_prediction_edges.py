"""Rotary positions, attention with decay and the loss over a table's rows at the edges
of what they take: the longest documents, extreme numbers, gradients nobody asked for."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import sparse_spatial_hashing_amd as ssh  # noqa: E402
import prediction_reference as ref  # noqa: E402
from test_gpu_prediction import _decay_case, _decay_compare, _loss_case, _on_gpu  # noqa: E402
from token_reference import check  # noqa: E402

DEV = torch.device("cuda:0")
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.mark.parametrize("reverse", [False, True])
def test_decay_the_longest_document(reverse):
    """As many tokens as a call takes, in the widest segments: the last one's end is near 2^31.

    All tokens are alike and a state falls by half: away from where a walk begins it is twice what a
    token adds."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 150 << 30:
        pytest.skip("needs 150 GiB")
    t = 2**31 - 4096
    one = lambda x: torch.tensor(x, dtype=BF16, device=DEV).view(1, 1, 8).expand(t, 1, 8)
    q, k, v, g = one([0.5] * 8), one([0.5] * 8), one([c / 4 for c in range(1, 9)]), one([1.0] * 8)
    decay = torch.tensor([math.log(2.0)], device=DEV)
    print(f"decay of {t} tokens, reverse {reverse}", flush=True)
    out, last, carry = ssh.decay_attend(q, k, v, decay, scale=1.0, reverse=reverse, return_carry=True)
    assert t // 65536 == carry.shape[0]
    value = v[0, 0].double().cpu()

    def alike(x, want, what):
        # away from both ends, and through the last segments
        for lo in (100, 2**30 - 50, t - 140000):
            for at in range(lo, min(lo + 139900, t - 100), 35000):
                part = x[at:min(at + 35000, t - 100)].cpu().double()
                # the state's copy, the result and some 2^-20 of sums
                assert ((part - want).abs() <= want.abs() * (2.0 ** -7)).all(), (what, at)

    alike(out, 4.0 * value, "out")
    assert ((last[0, 0].cpu().double() - value).abs() <= value * 2.0 ** -18).all()
    del out, last
    gq, gk, gv, gs = ssh.decay_attend_grad(g, q, k, v, decay, carry, scale=1.0, reverse=reverse)
    assert gs is None
    alike(gq, torch.full((8,), 9.0).double(), "gq")
    alike(gk, torch.full((8,), 9.0).double(), "gk")
    alike(gv, torch.full((8,), 4.0).double(), "gv")
    del gq, gk, gv
    torch.cuda.empty_cache()


def test_decay_an_unused_state_costs_nothing_in_the_backward():
    """The last state is returned and not used: no memory of its size, and the gradients are those without it."""
    gen = torch.Generator(device=DEV).manual_seed(1)
    docs, heads, width = 300, 4, 64
    at = torch.arange(docs + 1, dtype=torch.int32, device=DEV) * 40
    q, k, v, g = (torch.randn((40 * docs, heads, width), generator=gen, device=DEV).to(BF16) for _ in range(4))
    decay = torch.full((heads,), 0.1, device=DEV)
    size = 4 * docs * heads * width * width
    made = []
    for how in ("unused", "not returned"):
        leaves = [x.clone().requires_grad_() for x in (q, k, v)]
        out, last = ssh.decay_attend(*leaves, decay, at, return_state=how == "unused")
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        out.backward(g)
        peak = torch.cuda.max_memory_allocated() - before
        # the gradients, and the sums that the backward's own walk keeps: a row for each segment
        # but a document's last, and none of these has two
        rows = ssh.decay_attend(q, k, v, decay, at, return_carry=True)[2].shape[0]
        most = 3 * 2 * q.numel() + 4 * rows * heads * width * width + (1 << 20)
        assert peak <= most, (how, peak, most)
        assert most - 6 * q.numel() < size
        made.append([x.grad for x in leaves])
    assert all(torch.equal(a, b) for a, b in zip(*made))
    zero = torch.zeros((docs, heads, width, width), device=DEV)
    carry = ssh.decay_attend(q, k, v, decay, at, return_carry=True)[2]
    want = ssh.decay_attend_grad(g, q, k, v, decay, carry, at, grad_state=zero)
    assert all(torch.equal(a, b) for a, b in zip(made[0], want[:3]))


def test_decay_gradient_of_the_state_alone():
    gen = torch.Generator(device=DEV).manual_seed(2)
    q, k, v = (torch.randn((90, 2, 32), generator=gen, device=DEV).to(BF16).requires_grad_() for _ in range(3))
    state = torch.randn((1, 2, 32, 32), generator=gen, device=DEV).requires_grad_()
    decay, g = torch.full((2,), 0.05, device=DEV), torch.randn((1, 2, 32, 32), generator=gen, device=DEV)
    out, last, carry = ssh.decay_attend(q, k, v, decay, state=state, return_carry=True)
    made = torch.autograd.grad(last, (q, k, v, state), g)
    want = ssh.decay_attend_grad(torch.zeros_like(out), q.detach(), k.detach(), v.detach(), decay, carry,
                                 state=state.detach(), grad_state=g)
    assert not made[0].any() and all(torch.equal(a, b) for a, b in zip(made, want))
    (none,) = torch.autograd.grad(ssh.row_loss(q.flatten(1), k.flatten(1)[:50], torch.full((90,), -1, device=DEV)).sum(), q)
    assert not none.any()


@pytest.mark.parametrize("rate", [85.0, 42.0, 12.0])
@pytest.mark.parametrize("scale", [1.0, 1e-3])
def test_decay_fp16_weights_far_under_the_state(rate, scale):
    """A query that meets nothing of the nearest keys: its weights are of 2^-120 and less next to a
    state of thousands, of which e^-rate is left by the token and soon nothing. No inf by zero."""
    apart = max(1, round(84 / rate))  # tokens to the nearest key that a query meets
    t, width = 90, 16
    q, k = torch.zeros((t, 1, width), dtype=F16), torch.zeros((t, 1, width), dtype=F16)
    i = torch.arange(t)
    q[i, 0, i % 13] = 1.0
    k[i, 0, (i + apart) % 13] = 1.0  # q[i] meets k[i - apart], and every thirteenth before it
    gen = torch.Generator().manual_seed(3)
    s = dict(q=q, k=k, v=torch.randn((t, 1, width), generator=gen).to(F16), decay=torch.tensor([rate]),
             grad=torch.randn((t, 1, width), generator=gen).to(F16), state=torch.full((1, 1, width, width), 4000.0),
             grad_state=torch.full((1, 1, width, width), -3000.0))
    for reverse in (False, True):
        _decay_compare(s, [0, t], f"fp16 weights under the state, rate {rate} scale {scale}", reverse, scale)
    # queries of nothing next to a state near the largest number
    s["q"] = torch.zeros_like(q)
    g = {n: x.to(DEV) for n, x in s.items()}
    out, _ = ssh.decay_attend(g["q"], g["k"], g["v"], g["decay"], state=torch.full_like(g["state"], 3e38), scale=scale)
    assert not out.any()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("t,width", [(5, 64), (9, 200), (100, 32), (300, 128), (300, 200), (700, 72)])
def test_row_loss_rows_of_minus_infinity(dtype, t, width):
    """Rows ruled out by -inf against an element that is 1 in every token: their weights are 0, whatever
    tokens without a row, and the places past the last token, would make of such a row."""
    rows = 500
    x, table, ids, grad = _loss_case(t, rows, width, dtype, t + width, none=0.2)
    ids[0] = -1
    x[:, 0] = 1.0
    out = torch.zeros(rows, dtype=torch.bool)
    out[3::7] = True
    ids[(ids >= 0) & out[ids.clamp(min=0)]] -= 1
    left = (~out).cumsum(0) - 1
    few = torch.where(ids >= 0, left[ids.clamp(min=0)], -1)
    want = ref.row_loss(x, table[~out], few, 1.0, grad)
    table[out, 0] = -math.inf
    args = x.to(DEV), table.to(DEV), ids.to(DEV)
    print(f"row loss, rows of -inf, {dtype} {t} {width}", flush=True)
    loss, lse = ssh.row_loss(*args, return_lse=True)
    gx, gt = (v.cpu() for v in ssh.row_loss_grad(grad.to(DEV), *args, lse))
    check(loss, *want["loss"], "loss")
    check(lse, *want["lse"], "lse")
    check(gt[~out], *want["gt"], "gt")
    assert not gt[out].any()
    # element 0 of a token's gradient is 0 times -inf
    check(gx[:, 1:], *(v[:, 1:] for v in want["gx"]), "gx")
    assert not gx[ids < 0].any()


@pytest.mark.parametrize("t", [9, 300])
@pytest.mark.parametrize("size,scale", [(1e38, 4e4), (1e38, 1.0), (1e-38, 1.0), (1e-44, 1e30)])
def test_row_loss_fp16_gradients_at_the_ends_of_float32(t, size, scale):
    """The power of two that weights are taken up by may take scale past the largest float: elements
    that are 0 stay 0, what passes fp16's largest number is infinite, and none is NaN."""
    gen = torch.Generator().manual_seed(t)
    x, table = (torch.randn((n, 40), generator=gen) * min(1.0, scale ** -0.5) for n in (t, 70))
    if scale > 1e5:
        x, table = torch.zeros_like(x), torch.sign(table)  # no logits pass the largest float
    x[:, 5] = 0.0
    table[:, 5] = 0.0
    x, table, ids = x.half(), table.half(), torch.randint(0, 70, (t,), generator=gen)
    grad = torch.full((t,), size)
    want = ref.row_loss(x, table, ids, scale, grad)
    args = x.to(DEV), table.to(DEV), ids.to(DEV)
    print(f"row loss, gradients of {size} by {scale}", flush=True)
    loss, lse = ssh.row_loss(*args, scale=scale, return_lse=True)
    for n, v in zip(("gx", "gt"), ssh.row_loss_grad(grad.to(DEV), *args, lse, scale=scale)):
        value, bound = want[n]
        v = v.cpu().double()
        assert not v[:, 5].any() and not v.isnan().any(), n
        if size < 1 or scale == 1.0:
            over = value.abs() + bound > 65504
            assert (v[over] * value[over].sign() > 65504 - 2 * bound[over]).all(), n
            check(torch.where(over, 0, v), torch.where(over, 0, value), bound, n)


@pytest.mark.parametrize("dtype,t,rows,width", [(F16, 600_001, 300, 136), (BF16, 540_000, 260, 40),
                                                (BF16, 1_100_000, 60, 24), (F16, 524_289, 40, 8)])
def test_row_loss_bands_of_tokens(dtype, t, rows, width):
    """More tokens than 256 rows' weights are kept for at once (2^19): the table's gradient is summed over
    bands of them, a token's own over pieces of the rows."""
    x, table, ids, grad = _loss_case(t, rows, width, dtype, 41, size=1e-3)
    x, table, ids, grad = (v.to(DEV) for v in (x, table, ids, grad))
    x[ids < 0] = math.nan
    print(f"row loss, bands, {dtype} {t} {rows} {width}", flush=True)
    with torch.device(DEV):
        want = ref.row_loss(x, table, ids, 1.0, grad)
    loss, lse = ssh.row_loss(x, table, ids, return_lse=True)
    both = ssh.row_loss_grad(grad, x, table, ids, lse)
    for n, v in zip(("loss", "lse", "gx", "gt"), (loss, lse, *both)):
        value, bound = want[n]
        off = (v.double() - value).abs()
        assert (off <= bound).all(), (n, float((off / bound.clamp(min=1e-300)).nan_to_num(1e30).max()))
    del want
    for n in (0, 1):
        leaves = [x.clone(), table.clone()]
        leaves[n].requires_grad_()
        (made,) = torch.autograd.grad(ssh.row_loss(*leaves, ids), leaves[n], grad)
        assert torch.equal(made, both[n])


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("width,heads,kv_heads,lens", [
    (32, 2, 1, [20000, 3000]), (128, 1, 1, [9000, 40]), (64, 16, 4, [9000, 7011]), (40, 12, 6, [12000]),
    (64, 8, 8, [370 + 17 * (i % 20) for i in range(64)])])
def test_decay_gradients_of_longer_segments(dtype, reverse, width, heads, kv_heads, lens):
    """Segments of more than 128 tokens (the last case: twice as many as places, since documents end in them)."""
    s, at = _decay_case(lens, heads, kv_heads, width, dtype, 43, 5)
    g = {n: x.to(DEV) for n, x in s.items()}
    offsets = torch.tensor(at, dtype=torch.int32, device=DEV)
    print(f"decay, longer segments, {dtype} {len(lens)} documents, width {width} heads {heads}/{kv_heads}", flush=True)
    more = dict(state=g["state"], reverse=reverse)
    out, last, carry = ssh.decay_attend(g["q"], g["k"], g["v"], g["decay"], offsets, return_carry=True, **more)
    rows = carry.shape[0]
    assert s["q"].shape[0] // rows > 128, rows
    assert len(lens) < 64 or rows > 512 * 128 // width // heads  # doubled
    made = dict(zip(("gq", "gk", "gv", "gs"),
                    ssh.decay_attend_grad(g["grad"], g["q"], g["k"], g["v"], g["decay"], carry, offsets,
                                          grad_state=g["grad_state"], **more)), out=out, last=last)
    want = _on_gpu(ref.decay_attend, s["q"], s["k"], s["v"], s["decay"], at, width ** -0.5, s["state"], reverse,
                   s["grad"], s["grad_state"])
    for n, x in made.items():
        check(x, *want[n], n)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("width,heads,kv_heads", [(8, 2, 1), (32, 2, 2), (64, 2, 1), (128, 2, 2)])
def test_decay_long_documents_among_short_ones(dtype, reverse, width, heads, kv_heads):
    """Calls that go by one launch: documents of more than 256 tokens take several blocks there, each from
    the document's beginning on."""
    for lens, first, state in (([1] * 150 + [900] + [1] * 150 + [1], 0, True),
                               ([3, 0] * 100 + [257, 256, 513, 258, 0] + [4] * 60, 7, False),
                               ([0] * 300 + [1283], 2, True)):
        s, at = _decay_case(lens, heads, kv_heads, width, dtype, 47, first, state)
        made = _decay_compare(s, at, f"decay, long ones among short, {dtype} {len(lens)} width {width}", reverse)
        carry = ssh.decay_attend(*(s[n].to(DEV) for n in "qkv"), s["decay"].to(DEV),
                                 torch.tensor(at, dtype=torch.int32, device=DEV), return_carry=True)[2]
        assert carry.shape[0] == 0
        # the same inputs give the same bits
        again = _decay_compare(s, at, "again", reverse)
        assert all(made[n] is None or torch.equal(made[n], again[n]) for n in made)


@pytest.mark.parametrize("how", ["rising and back", "falling", "past the end", "jumps", "right"])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("heads,kv_heads,width", [(2, 1, 32), (2, 2, 72)])
def test_decay_one_launch_writes_nothing_outside(how, reverse, heads, kv_heads, width):
    """Wrong offsets of calls that go by one launch, with every output inside a fence."""
    from sparse_spatial_hashing_amd import prediction
    from test_gpu_token_paths import Fenced
    lib, stream = prediction._lib, torch.cuda.current_stream().cuda_stream
    t, docs = 1100, 600
    gen = torch.Generator(device=DEV).manual_seed(5)
    jumps = torch.randint(-50, t + 50, (docs + 1,), generator=torch.Generator().manual_seed(6)).tolist()
    ends = {"rising and back": [0] * 200 + [t] * 200 + [300] * 201, "falling": [t - 2 * i for i in range(docs + 1)],
            "past the end": [-2**31] * 100 + [5] * 200 + [2**31 - 1] * 301, "jumps": jumps,
            "right": list(range(300)) + [t - 300 + i for i in range(301)]}[how]
    q, k, v, g = (torch.randn((t, h, width), generator=gen, device=DEV).to(BF16)
                  for h in (heads, kv_heads, kv_heads, heads))
    shape = (docs, heads, width, width)
    state, gl = (torch.randn(shape, generator=gen, device=DEV) for _ in range(2))
    decay, offsets = torch.full((heads,), 0.01, device=DEV), torch.tensor(ends, dtype=torch.int32, device=DEV)
    a, kept, _ = prediction._decay_args(q, k, v, decay, offsets, None, reverse, g)
    assert lib.tok_decay_carry_rows(a) == 0
    f = Fenced()
    out, last = f.take(q.shape, BF16), f.take(shape, F32)
    print(f"fenced decay in one launch, {how} reverse {reverse} width {width}", flush=True)
    assert lib.tok_decay_attend(a, q.data_ptr(), k.data_ptr(), v.data_ptr(), state.data_ptr(), out.data_ptr(),
                                last.data_ptr(), None, stream) == 0
    f.check()
    nbytes = lib.tok_decay_grad_workspace_bytes(a)
    ws, made = f.take((nbytes,), torch.uint8) if nbytes else None, [f.take(x.shape, BF16) for x in (q, k, v)]
    gs = f.take(shape, F32)
    assert lib.tok_decay_attend_grad(a, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), state.data_ptr(), None,
                                     gl.data_ptr(), *[x.data_ptr() for x in made], gs.data_ptr(),
                                     None if ws is None else ws.data_ptr(), nbytes, stream) == 0
    f.check()
    if how == "right":
        m = dict(state=state, reverse=reverse)
        want = ssh.decay_attend(q, k, v, decay, offsets, return_carry=True, **m)
        grads = ssh.decay_attend_grad(g, q, k, v, decay, want[2], offsets, grad_state=gl, **m)
        for x, y in zip((out, last, *made, gs), (*want[:2], *grads)):
            assert torch.equal(x, y)


def test_rotate_far_and_fast():
    """The turn is right to 2^-25 wherever it is: positions and frequencies of 2^31 turns and far more, against
    their exact product."""
    from decimal import Decimal, getcontext
    getcontext().prec = 60
    whole = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")
    freqs = [1.0, 3.0, 10.0, 0.1, 1e-4, 1234.5678, 1e6 / 3]
    positions = [2**31 - 1, -2**31, 2**31 - 2, 1987654321, -1234567891, 2**30 + 1, 99991, -1, 0]
    x = torch.zeros((len(positions), 1, 2 * len(freqs)), device=DEV)
    x[..., :len(freqs)] = 1.0
    got = ssh.rotate(x, torch.tensor(positions, dtype=torch.int32, device=DEV),
                     torch.tensor([freqs], dtype=torch.float64, device=DEV)).cpu().double()[:, 0]
    # the turn, two steps of a sine near 1, and the products'
    bound = 2 * math.pi * 2.0 ** -25 + 4 * 2.0 ** -24
    for i, p in enumerate(positions):
        for j, f in enumerate(freqs):
            turns = Decimal(p) * Decimal(f) / whole
            angle = float((turns - turns.to_integral_value()) * whole)
            assert abs(got[i, j] - math.cos(angle)) <= bound, (p, f)
            assert abs(got[i, len(freqs) + j] - math.sin(angle)) <= bound, (p, f)


def test_graphs_of_long_documents_and_bands():
    from test_gpu_tokens import _replays
    s, at = _decay_case([1] * 200 + [700] + [2] * 100, 2, 1, 64, BF16, 53)
    g, offsets = {n: x.to(DEV) for n, x in s.items()}, torch.tensor(at, dtype=torch.int32, device=DEV)
    x, table, ids, grad = (v.to(DEV) for v in _loss_case(524_300, 40, 8, BF16, 59))

    def step():
        out, last, carry = ssh.decay_attend(g["q"], g["k"], g["v"], g["decay"], offsets, state=g["state"],
                                            return_carry=True)
        grads = ssh.decay_attend_grad(g["grad"], g["q"], g["k"], g["v"], g["decay"], carry, offsets, state=g["state"],
                                      grad_state=g["grad_state"])
        loss, lse = ssh.row_loss(x, table, ids, return_lse=True)
        return (out, last, *grads, loss, *ssh.row_loss_grad(grad, x, table, ids, lse))

    _replays(step, [g["q"], g["k"], g["v"], g["grad"], g["state"], x, table, grad])


def test_two_streams_at_once():
    """The same operators on two streams over the same tensors, workspaces of their own."""
    s, at = _decay_case([1] * 200 + [900] + [2] * 100, 2, 1, 64, BF16, 61)
    g, offsets = {n: x.to(DEV) for n, x in s.items()}, torch.tensor(at, dtype=torch.int32, device=DEV)
    x, table, ids, grad = (v.to(DEV) for v in _loss_case(3000, 5000, 136, F16, 67))

    def run():
        made = ssh.decay_attend(g["q"], g["k"], g["v"], g["decay"], offsets, state=g["state"], return_carry=True)
        grads = ssh.decay_attend_grad(g["grad"], g["q"], g["k"], g["v"], g["decay"], made[2], offsets, state=g["state"])
        loss, lse = ssh.row_loss(x, table, ids, return_lse=True)
        return (*made[:2], *grads, loss, *ssh.row_loss_grad(grad, x, table, ids, lse))

    want = run()
    sides, made = [torch.cuda.Stream() for _ in range(2)], []
    for side in sides:
        side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for side in sides:
            with torch.cuda.stream(side):
                made.append(run())
    torch.cuda.synchronize()
    for got in made:
        assert all(torch.equal(a, b) for a, b in zip(got, want))
