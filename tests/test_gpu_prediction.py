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
            check(x, *want[n], f"{what} {n}")
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
