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
