"""Rotary positions, attention with decay and the loss over a table's rows without a
GPU: the 64-bit reference against differences, frequencies, and the refusals, which
come before any GPU call."""
import ctypes
import math

import pytest
import torch
import torch.autograd.forward_ad as forward_ad
from torch.fx.experimental.proxy_tensor import make_fx

import prediction_reference as ref
import sparse_spatial_hashing_amd as ssh
from sparse_spatial_hashing_amd import prediction
from test_tokens_cpu import _numbers
from token_reference import check

LIB = prediction._lib
EINVAL, EWORKSPACE = -1, -2


# ------------------------------------------------------------------ reference --

def test_reference_loss_gradient_by_differences():
    gen = torch.Generator().manual_seed(1)
    x, table = torch.randn((5, 3), generator=gen, dtype=torch.float64), torch.randn((4, 3), generator=gen,
                                                                                    dtype=torch.float64)
    ids, grad = torch.tensor([2, -1, 0, 2, 4]), torch.randn(5, generator=gen, dtype=torch.float64)
    made = ref.row_loss(x, table, ids, 0.7, grad)

    def total():
        return float((ref.row_loss(x, table, ids, 0.7)["loss"][0] * grad).sum())

    for name, t in (("gx", x), ("gt", table)):
        assert torch.allclose(made[name][0], _numbers(total, t), rtol=0, atol=1e-7), name
    assert not made["loss"][0][[1, 4]].any() and not made["gx"][0][[1, 4]].any()


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("with_state", [False, True])
def test_reference_decay_gradient_by_differences(reverse, with_state):
    gen = torch.Generator().manual_seed(2)
    at, heads = [0, 3, 3, 5], 2
    q, k, v, g = (torch.randn((5, h, 2), generator=gen, dtype=torch.float64) for h in (heads, 1, 1, heads))
    decay = torch.tensor([0.3, 0.0])
    state, gl = (torch.randn((3, heads, 2, 2), generator=gen, dtype=torch.float64) if with_state else None
                 for _ in range(2))

    def total():
        r = ref.decay_attend(q, k, v, decay, at, 0.6, state, reverse)
        return float((r["out"][0] * g).sum()) + (float((r["last"][0] * gl).sum()) if with_state else 0.0)

    made = ref.decay_attend(q, k, v, decay, at, 0.6, state, reverse, g, gl)
    for name, t in (("gq", q), ("gk", k), ("gv", v), ("gs", state)):
        if t is not None:
            assert torch.allclose(made[name][0], _numbers(total, t), rtol=0, atol=1e-6), name


@pytest.mark.parametrize("reverse", [False, True])
def test_reference_decay_is_its_recurrence(reverse):
    gen = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn((6, 1, 3), generator=gen, dtype=torch.float64) for _ in range(3))
    state = torch.randn((1, 1, 3, 3), generator=gen, dtype=torch.float64)
    made = ref.decay_attend(q, k, v, torch.tensor([0.25]), [0, 6], 2.0, state, reverse)
    s = state[0, 0]
    for t in reversed(range(6)) if reverse else range(6):
        s = math.exp(-0.25) * s + k[t, 0][:, None] * v[t, 0][None]
        assert torch.allclose(made["out"][0][t, 0], 2.0 * q[t, 0] @ s)
    assert torch.allclose(made["last"][0][0, 0], s)


@pytest.mark.parametrize("interleaved", [False, True])
def test_reference_rotation_turns_back_and_keeps_lengths(interleaved):
    gen = torch.Generator().manual_seed(4)
    x = torch.randn((9, 2, 14), generator=gen, dtype=torch.float64)
    pos = torch.randint(-50, 50, (9, 3), generator=gen, dtype=torch.int32)
    freqs = ssh.rotary_frequencies(12, axes=3, device="cpu")
    out = ref.rotate(x, pos, freqs, interleaved)[0]
    assert torch.allclose(ref.rotate(out, pos, freqs, interleaved, True)[0], x)
    assert torch.allclose(out.norm(dim=2), x.norm(dim=2)) and torch.equal(out[..., 12:], x[..., 12:])
    # a turn of two tokens' positions by the same places leaves their products as they were
    moved = ref.rotate(x, pos + 17, freqs, interleaved)[0]
    assert torch.allclose(out[0, 0] @ out[1, 0],
                          (ref.rotate(x, pos + 17, freqs, interleaved)[0][0, 0] @ moved[1, 0]))


def test_planted_mistakes_are_seen():
    """The bounds are tight enough for a token too many, a decay too few, a row too many."""
    gen = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn((40, 1, 32), generator=gen).to(torch.bfloat16) for _ in range(3))
    good = ref.decay_attend(q, k, v, torch.tensor([0.1]), [0, 40], 0.2)
    for name, wrong in (("out", ref.decay_attend(q, k, v, torch.tensor([0.09]), [0, 40], 0.2)),
                        ("out", ref.decay_attend(q, k, v, torch.tensor([0.1]), [0, 39, 40], 0.2)),
                        ("last", ref.decay_attend(q, k.roll(1, 0), v.roll(1, 0), torch.tensor([0.1]), [0, 40], 0.2))):
        with pytest.raises(AssertionError):
            check(wrong[name][0], *good[name], "planted")
    x, table = torch.randn((6, 16), generator=gen).to(torch.bfloat16), torch.randn((90, 16), generator=gen).to(torch.bfloat16)
    ids, g = torch.randint(0, 89, (6,), generator=gen), torch.ones(6)
    good, wrong = ref.row_loss(x, table, ids, 0.5, g), ref.row_loss(x, table[:89], ids, 0.5, g)
    for name in ("loss", "lse", "gx"):
        with pytest.raises(AssertionError):
            check(wrong[name][0], *good[name], "planted")
    pos, freqs = torch.arange(6, dtype=torch.int32) + 1, ssh.rotary_frequencies(16, device="cpu")
    with pytest.raises(AssertionError):
        check(ref.rotate(x[:, None], pos + 1, freqs)[0], *ref.rotate(x[:, None], pos, freqs), "planted")


# ---------------------------------------------------------------- frequencies --

def test_frequencies():
    f = ssh.rotary_frequencies(8, device="cpu")
    assert f.dtype == torch.float64 and f.shape == (1, 4)
    assert torch.allclose(f[0], torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64))
    f = ssh.rotary_frequencies(12, axes=3, base=100.0, device="cpu")
    assert f.shape == (3, 2) and torch.equal(f[0], f[2]) and torch.allclose(f[0, 1], torch.tensor(0.1).double())
    assert torch.allclose(ssh.rotary_frequencies(8, stretch=4.0, device="cpu"), ssh.rotary_frequencies(8, device="cpu") / 4)
    plain, long = (ssh.rotary_frequencies(64, device="cpu", **m)[0] for m in (dict(), dict(stretch=8.0, context=4096)))
    turns = 4096 * plain / (2 * math.pi)
    assert torch.equal(long[turns >= 32], plain[turns >= 32]) and torch.allclose(long[turns <= 1], plain[turns <= 1] / 8)
    between = (turns > 1) & (turns < 32)
    assert between.any() and (long[between] < plain[between]).all() and (long[between] > plain[between] / 8).all()
    assert (long[1:] < long[:-1]).all()


@pytest.mark.parametrize("bad", [dict(rotated=7), dict(rotated=8, axes=3), dict(rotated=0), dict(rotated=8, axes=0),
                                 dict(rotated=8, axes=4), dict(rotated=8, base=0.0), dict(rotated=8, base=math.inf),
                                 dict(rotated=8, stretch=0.5), dict(rotated=8, stretch=math.nan),
                                 dict(rotated=8, context=-1), dict(rotated=8, turns=(4.0, 2.0))])
def test_frequencies_refuse(bad):
    with pytest.raises(ValueError):
        ssh.rotary_frequencies(device="cpu", **bad)


# ------------------------------------------------------------------- refusals --

HALF = torch.zeros((4, 1, 8), dtype=torch.bfloat16)
ROWS, IDS = torch.zeros((4, 8), dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
RATE, LOSS, STATE = torch.zeros(1), torch.zeros(4), torch.zeros((1, 1, 8, 8))
CARRY, FREQS = torch.zeros((0, 1, 8, 8)), torch.zeros((1, 4), dtype=torch.float64)
CALLS = {
    "rotate": (HALF, lambda t: ssh.rotate(t, IDS, FREQS)),
    "rotate freqs": (FREQS, lambda t: ssh.rotate(HALF, IDS, t)),
    "decay_attend q": (HALF, lambda t: ssh.decay_attend(t, HALF, HALF, RATE)[0]),
    "decay_attend v": (HALF, lambda t: ssh.decay_attend(HALF, HALF, t, RATE)[0]),
    "decay_attend decay": (RATE, lambda t: ssh.decay_attend(HALF, HALF, HALF, t)[0]),
    "decay_attend state": (STATE, lambda t: ssh.decay_attend(HALF, HALF, HALF, RATE, state=t)[0]),
    "decay_attend_grad": (HALF, lambda t: ssh.decay_attend_grad(t, HALF, HALF, HALF, RATE, CARRY)[0]),
    "row_loss x": (ROWS, lambda t: ssh.row_loss(t, ROWS, IDS)),
    "row_loss table": (ROWS, lambda t: ssh.row_loss(ROWS, t, IDS)),
    "row_loss_grad": (LOSS, lambda t: ssh.row_loss_grad(t, ROWS, ROWS, IDS, LOSS)[0]),
}


@pytest.mark.parametrize("name", CALLS)
def test_cpu_tensors_and_tangents_are_refused(name):
    t, call = CALLS[name]
    with pytest.raises(ValueError, match="GPU"):
        call(t)
    with forward_ad.dual_level():
        with pytest.raises(NotImplementedError, match="forward-mode"):
            call(forward_ad.make_dual(t, torch.ones_like(t)))


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("how", [dict(), dict(pre_dispatch=True), dict(tracing_mode="fake"), "jit"])
def test_tracing_is_refused(name, how):
    t, call = CALLS[name]
    with pytest.raises(NotImplementedError, match="traced"):
        if how == "jit":
            torch.jit.trace(call, t)
        else:
            make_fx(call, **how)(t)


def test_constants_that_want_gradients_are_refused():
    with pytest.raises(ValueError, match="constant"):
        ssh.decay_attend(HALF, HALF, HALF, RATE.clone().requires_grad_())
    with pytest.raises(ValueError, match="constant"):
        ssh.rotate(HALF, IDS, FREQS.clone().requires_grad_())
    with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
        ssh.decay_attend(HALF, HALF, HALF, RATE.clone().requires_grad_())


def test_rotation_refuses():
    p = 4096  # never read: the call returns first
    good = [p, 10, 4, 64, 256, 64, 1, p, 2, 1, 2, p, 8, 0, 0, p, None]
    for i, bad in ((1, -1), (1, 2**31), (2, 0), (2, 65537), (3, 0), (3, 31), (3, 65537), (4, -1), (5, -1), (6, 3),
                   (6, -1), (8, -1), (9, -1), (10, 0), (10, 4), (12, 0), (12, 17), (13, 2), (14, -1), (0, None),
                   (7, None), (11, None), (15, None), (0, p + 1), (7, p + 2), (11, p + 4), (15, p + 1)):
        args = list(good)
        args[i] = bad
        assert LIB.tok_rotate(*args) == EINVAL, (i, bad)
    assert LIB.tok_rotate(None, 0, *good[2:7], None, 2, 1, 2, None, 8, 0, 0, None, None) == 0  # no tokens


def test_loss_refuses():
    p = 4096
    for t, rows, width in ((-1, 4, 8), (2**25 + 1, 4, 8), (4, 0, 8), (4, 2**31 - 2047, 8), (4, 4, 0), (4, 4, 12),
                           (4, 4, 65544)):
        assert LIB.tok_row_loss_workspace_bytes(t, rows, width) == EINVAL
        assert LIB.tok_row_loss_grad_workspace_bytes(t, rows, width) == EINVAL
    for t, rows, width in ((2**25, 4, 8), (4, 2**31 - 2048, 8), (4, 4, 65536), (1, 1, 8)):
        assert LIB.tok_row_loss_workspace_bytes(t, rows, width) > 0
        assert LIB.tok_row_loss_grad_workspace_bytes(t, rows, width) > 0
    nbytes = LIB.tok_row_loss_workspace_bytes(100, 50, 16)
    good = [p, 16, p, 16, 1, 100, 50, 16, p, 4, 1.0, p, p, p, nbytes, None]
    for i, bad in ((0, None), (0, p + 8), (1, -8), (1, 12), (1, 2**22), (2, None), (2, p + 2), (3, -8), (3, 2**22),
                   (3, 4), (4, 0), (4, 3), (5, -1), (6, 0), (7, 12), (8, None), (8, p + 2), (9, 2), (10, 0.0),
                   (10, -1.0), (10, math.inf), (10, math.nan), (11, None), (11, p + 2), (12, p + 1)):
        args = list(good)
        args[i] = bad
        assert LIB.tok_row_loss(*args) == EINVAL, (i, bad)
    for i, bad in ((13, None), (13, p + 64), (14, nbytes - 1)):
        args = list(good)
        args[i] = bad
        assert LIB.tok_row_loss(*args) == EWORKSPACE, (i, bad)
    nbytes = LIB.tok_row_loss_grad_workspace_bytes(100, 50, 16)
    good = [p, p, 16, p, 16, 1, 100, 50, 16, p, 8, p, 1.0, p, p, p, nbytes, None]
    for i, bad in ((0, None), (0, p + 2), (1, None), (2, 12), (3, None), (4, 2**22), (5, 0), (6, -1), (7, 0), (8, 4),
                   (9, None), (9, p + 4), (10, 3), (11, None), (12, 0.0), (13, p + 8), (14, p + 2)):
        args = list(good)
        args[i] = bad
        assert LIB.tok_row_loss_grad(*args) == EINVAL, (i, bad)
    args = list(good)
    args[13] = args[14] = None  # one gradient or both
    assert LIB.tok_row_loss_grad(*args) == EINVAL
    for i, bad in ((15, None), (15, p + 64), (16, nbytes - 1)):
        args = list(good)
        args[i] = bad
        assert LIB.tok_row_loss_grad(*args) == EWORKSPACE, (i, bad)
    # the largest pieces of a call stay in the cache between memory and the XCDs
    assert LIB.tok_row_loss_grad_workspace_bytes(4096, 214272, 512) < 1 << 30


def _decay(**more):
    base = dict(dtype=1, heads=4, kv_heads=2, width=64, t=8000, docs=1, reverse=0, decay=4096, scale=1.0,
                q_stride=(256, 64), k_stride=(128, 64), v_stride=(128, 64), g_stride=(256, 64))
    base.update(more)
    return ctypes.byref(prediction._Decay(**base))


@pytest.mark.parametrize("bad", [
    dict(dtype=0), dict(dtype=3), dict(heads=3), dict(heads=0), dict(kv_heads=0), dict(heads=65538), dict(width=0),
    dict(width=12), dict(width=136), dict(t=-1), dict(t=2**31 - 4095, heads=1, kv_heads=1), dict(t=2**30), dict(docs=0),
    dict(docs=2), dict(docs=2**20 + 1, offsets=16), dict(docs=2**20, offsets=16, heads=1024, kv_heads=1024),
    dict(reverse=2), dict(decay=None), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.inf), dict(scale=math.nan),
    dict(reserved=1), dict(q_stride=(255, 64)), dict(k_stride=(128, 4)), dict(v_stride=(-128, 64)),
    dict(k_stride=(2**25, 64))])
def test_decay_refuses(bad):
    a, p = _decay(**bad), 4096
    assert LIB.tok_decay_carry_rows(a) == EINVAL and LIB.tok_decay_grad_workspace_bytes(a) == EINVAL
    assert LIB.tok_decay_attend(a, p, p, p, p, p, p, p, None) == EINVAL
    assert LIB.tok_decay_attend_grad(a, *[p] * 12, 1 << 40, None) == EINVAL


def test_decay_refuses_pointers_and_workspaces():
    a, p = _decay(), 4096
    assert LIB.tok_decay_carry_rows(None) == EINVAL
    assert LIB.tok_decay_carry_rows(a) > 0  # segments, whose states are kept
    good = [p] * 7
    for i in (0, 1, 2, 4, 6):  # q, k, v, out, carry
        assert LIB.tok_decay_attend(a, *[None if j == i else x for j, x in enumerate(good)], None) == EINVAL, i
    for i in range(7):
        assert LIB.tok_decay_attend(a, *[p + 8 if j == i else x for j, x in enumerate(good)], None) == EINVAL, i
    nbytes = LIB.tok_decay_grad_workspace_bytes(a)
    assert nbytes > 0
    good = [p] * 12
    for i in (0, 1, 2, 3, 5, 7, 8, 9):  # q, k, v, grad_out, carry, the gradients
        args = [None if j == i else x for j, x in enumerate(good)]
        assert LIB.tok_decay_attend_grad(a, *args, nbytes, None) == EINVAL, i
    for i in range(11):
        args = [p + 4 if j == i else x for j, x in enumerate(good)]
        assert LIB.tok_decay_attend_grad(a, *args, nbytes, None) == EINVAL, i
    for ws, n in ((None, nbytes), (p + 64, nbytes), (p, nbytes - 1)):
        assert LIB.tok_decay_attend_grad(a, *good[:11], ws, n, None) == EWORKSPACE
    assert LIB.tok_decay_attend_grad(_decay(g_stride=(3, 64)), *good, nbytes, None) == EINVAL


def test_decay_keeps_states_only_for_documents_of_several_segments():
    for more in (dict(t=0), dict(t=1), dict(t=64, docs=64, offsets=16), dict(t=128), dict(t=8000, docs=500, offsets=16),
                 dict(t=2**13, docs=2**12, offsets=16)):
        assert LIB.tok_decay_carry_rows(_decay(**more)) == 0, more
    for more in (dict(t=300), dict(t=20000), dict(t=20000, docs=500, offsets=16), dict(t=2**29 - 4096),
                 dict(t=2**21, docs=2**20, offsets=16)):
        assert 0 < LIB.tok_decay_carry_rows(_decay(**more)) <= more["t"] // 128, more
