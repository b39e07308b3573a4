"""Token operators without a GPU: the 64-bit reference against differences,
and the refusals, which come before any GPU call."""
import ctypes
import math

import pytest
import torch

import sparse_spatial_hashing_amd as ssh
import token_reference as ref
from sparse_spatial_hashing_amd import tokens

LIB = tokens._lib
EINVAL, EWORKSPACE = -1, -2


def _numbers(f, x, step=1e-6):
    """The gradient of the number f() by central differences in every element of x."""
    out = torch.zeros_like(x)
    for i in range(x.numel()):
        old = x.reshape(-1)[i].item()
        x.view(-1)[i] = old + step
        up = f()
        x.view(-1)[i] = old - step
        out.view(-1)[i] = (up - f()) / (2 * step)
        x.view(-1)[i] = old
    return out


@pytest.mark.parametrize("cap,axes,mask", [(0.0, 0, "full"), (1.5, 2, "causal"), (0.0, 3, "prefix")])
def test_reference_attention_gradient_by_differences(cap, axes, mask):
    gen = torch.Generator().manual_seed(3)
    q_at, k_at, heads = [0, 2, 2, 5], [0, 3, 4, 6], 2
    q, k, v, g = (torch.randn((n, h, 3), generator=gen, dtype=torch.float64)
                  for n, h in ((5, heads), (6, 1), (6, 1), (5, heads)))
    more = dict(q_at=q_at, k_at=k_at, scale=0.7, cap=cap, causal=mask == "causal",
                prefix=[2, 0, 1] if mask == "prefix" else None)
    if axes:
        more.update(slopes=torch.tensor([0.25, 0.0625]),
                    q_pos=torch.randint(0, 5, (5, axes), generator=gen),
                    k_pos=torch.randint(0, 5, (6, axes), generator=gen))
    made = ref.attend(q, k, v, grad=g, **more)
    for name, x in (("gq", q), ("gk", k), ("gv", v)):
        want = _numbers(lambda: float((ref.attend(q, k, v, **more)["out"][0] * g).sum()), x)
        assert torch.allclose(made[name][0], want, rtol=0, atol=1e-7), name


@pytest.mark.parametrize("reverse", [False, True])
def test_reference_recurrence_gradient_by_differences(reverse):
    gen = torch.Generator().manual_seed(4)
    at = [0, 4, 4, 5]
    gate, x, g = (torch.randn((5, 2), generator=gen, dtype=torch.float64) for _ in range(3))
    state, gl = (torch.randn((3, 2), generator=gen, dtype=torch.float64) for _ in range(2))

    def total():
        r = ref.scan(gate, x, at, state, reverse)
        return float((r["y"][0] * g).sum() + (r["last"][0] * gl).sum())

    made = ref.scan(gate, x, at, state, reverse, grad=g, grad_state=gl)
    for name, t in (("gg", gate), ("gx", x), ("gs", state)):
        assert torch.allclose(made[name][0], _numbers(total, t), rtol=0, atol=1e-7), name


def test_reference_embedding_gradient_by_differences():
    gen = torch.Generator().manual_seed(5)
    table, ids = torch.randn((4, 3), generator=gen, dtype=torch.float64), torch.tensor([1, -1, 3, 1, 4])
    g = torch.randn((5, 3), generator=gen, dtype=torch.float64)
    want = _numbers(lambda: float((ref.embed(table, ids, 1.5)[0] * g).sum()), table)
    assert torch.allclose(ref.embed_grad(g, ids, 4, 1.5)[0], want, rtol=0, atol=1e-7)


def test_a_wrong_weight_is_seen():
    """The bound is tight enough to see one key too many."""
    gen = torch.Generator().manual_seed(6)
    q, k, v = (torch.randn((40, 1, 32), generator=gen).to(torch.bfloat16) for _ in range(3))
    good = ref.attend(q, k, v, [0, 40], [0, 40], 0.2, causal=True)["out"]
    late = ref.attend(q, k, v, [0, 40], [0, 40], 0.2, prefix=[20])["out"]
    with pytest.raises(AssertionError):
        ref.check(late[0], *good, "planted")


# ------------------------------------------------------------------- refusals --

def test_cpu_tensors_are_refused():
    x = torch.zeros((4, 8))
    h = torch.zeros((4, 1, 8), dtype=torch.bfloat16)
    ids = torch.zeros(4, dtype=torch.int32)
    for call in (lambda: ssh.embed(x, ids), lambda: ssh.embed_grad(x, ids, 4),
                 lambda: ssh.attend(h, h, h), lambda: ssh.attend_grad(h, h, h, h, h, x[:, :1]),
                 lambda: ssh.gated_scan(x, x), lambda: ssh.gated_scan_grad(x, x, x, x)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(TypeError):
        ssh.embed([1.0], ids)


def _attention(**more):
    base = dict(dtype=1, heads=4, kv_heads=2, width=64, tq=8, tk=8, docs=1, mask=0, scale=1.0, cap=0.0,
                q_stride=(256, 64), k_stride=(128, 64), v_stride=(128, 64), g_stride=(256, 64))
    base.update(more)
    return tokens._Attention(**base)


@pytest.mark.parametrize("bad", [
    dict(dtype=0), dict(dtype=3), dict(heads=3), dict(heads=0), dict(kv_heads=0), dict(width=0),
    dict(width=12), dict(width=136), dict(tq=-1), dict(tk=2**31), dict(docs=0), dict(docs=2),
    dict(docs=2**20 + 1), dict(mask=2), dict(prefix=16), dict(scale=0.0), dict(scale=-1.0),
    dict(scale=math.inf), dict(scale=math.nan), dict(cap=-1.0), dict(cap=math.nan), dict(axes=4),
    dict(axes=1), dict(axes=2, slopes=16, q_pos=16), dict(reserved=1), dict(q_stride=(255, 64)),
    dict(k_stride=(128, 4)), dict(v_stride=(-128, 64)), dict(tq=2**30, heads=4)])
def test_attention_refuses(bad):
    a = ctypes.byref(_attention(**bad))
    p = 4096  # never read: the call returns first
    assert LIB.tok_attend_workspace_bytes(a) == EINVAL
    assert LIB.tok_attend_grad_workspace_bytes(a) == EINVAL
    assert LIB.tok_attend(a, p, p, p, p, None, p, 1 << 40, None) == EINVAL
    assert LIB.tok_attend_grad(a, *[p] * 10, 1 << 40, None) == EINVAL


def test_attention_refuses_pointers_and_workspaces():
    a, p = ctypes.byref(_attention()), 4096
    assert LIB.tok_attend_workspace_bytes(a) >= 0
    for q, k, v, o in ((None, p, p, p), (p, None, p, p), (p, p, None, p), (p, p, p, None),
                       (p + 8, p, p, p), (p, p, p + 2, p)):
        assert LIB.tok_attend(a, q, k, v, o, None, p, 1 << 40, None) == EINVAL
    nbytes = LIB.tok_attend_grad_workspace_bytes(a)
    args = [p] * 9
    assert nbytes > 0
    assert LIB.tok_attend_grad(a, *args, None, nbytes, None) == EWORKSPACE
    assert LIB.tok_attend_grad(a, *args, p + 64, nbytes, None) == EWORKSPACE
    assert LIB.tok_attend_grad(a, *args, p, nbytes - 1, None) == EWORKSPACE
    for i in range(9):
        bad = list(args)
        bad[i] = None
        assert LIB.tok_attend_grad(a, *bad, p, nbytes, None) == EINVAL, i
    odd = ctypes.byref(_attention(g_stride=(3, 64)))
    assert LIB.tok_attend_grad(odd, *args, p, nbytes, None) == EINVAL
    assert LIB.tok_attend_workspace_bytes(None) == EINVAL


def test_embedding_refuses():
    p = 4096
    good = [p, 10, 8, 8, 0, p, 4, 5, 1.0, p, None]
    for i, bad in ((1, 0), (1, 2**31), (2, 0), (2, 65537), (3, -1), (4, 3), (6, 2), (7, -1), (7, 2**31),
                   (0, None), (5, None), (9, None), (0, p + 1), (5, p + 2), (9, p + 2)):
        args = list(good)
        args[i] = bad
        assert LIB.tok_embed(*args) == EINVAL, (i, bad)
    assert LIB.tok_embed_grad_workspace_bytes(-1, 4, 4) == EINVAL
    assert LIB.tok_embed_grad_workspace_bytes(4, 0, 4) == EINVAL
    assert LIB.tok_embed_grad_workspace_bytes(4, 2**24 + 1, 4) == EINVAL
    assert LIB.tok_embed_grad_workspace_bytes(2**27 + 1, 4, 4) == EINVAL
    assert LIB.tok_embed_grad_workspace_bytes(5, 10, 8) == 0  # a few tokens need none
    nbytes = LIB.tok_embed_grad_workspace_bytes(5000, 10, 8)
    good = [p, 8, 0, p, 4, 5000, 10, 8, 1.0, p, p, nbytes, None]
    for i, bad in ((1, -1), (2, 9), (4, 3), (5, -1), (6, 0), (7, 0), (0, None), (3, None), (9, None),
                   (0, p + 2), (3, p + 2), (9, p + 8)):
        args = list(good)
        args[i] = bad
        assert LIB.tok_embed_grad(*args) == EINVAL, (i, bad)
    for i, bad in ((10, None), (10, p + 4), (11, nbytes - 1)):
        args = list(good)
        args[i] = bad
        assert LIB.tok_embed_grad(*args) == EWORKSPACE, (i, bad)


def test_recurrence_refuses():
    p = 4096
    assert LIB.tok_scan_runs(-1) == EINVAL and LIB.tok_scan_runs(2**31) == EINVAL
    run = tokens.TOK_SCAN_RUN
    assert [LIB.tok_scan_runs(n) for n in (0, 1, run, run + 1)] == [0, 1, 1, 2]
    assert LIB.tok_scan_workspace_bytes(4, 0) == EINVAL
    assert LIB.tok_scan_workspace_bytes(-1, 4) == EINVAL
    nbytes = LIB.tok_scan_workspace_bytes(5000, 8)
    good = [p, p, 0, 5000, 8, p, 2, 0, p, p, p, p, p, nbytes, None]
    for i, bad in ((2, 3), (3, -1), (3, 2**31), (4, 0), (4, 65537), (5, None), (6, 0), (6, 2**20 + 1),
                   (7, 2), (0, None), (1, None), (9, None)):
        args = list(good)
        args[i] = bad
        assert LIB.tok_scan(*args) == EINVAL, (i, bad)
    for i, bad in ((12, None), (12, p + 8), (13, nbytes - 1)):
        args = list(good)
        args[i] = bad
        assert LIB.tok_scan(*args) == EWORKSPACE, (i, bad)
    good = [p, p, p, p, 0, 5000, 8, p, 2, 0, p, p, p, p, p, p, nbytes, None]
    for i, bad in ((4, 3), (5, -1), (6, 0), (7, None), (8, 0), (9, 3), (0, None), (1, None), (2, None),
                   (3, None), (12, None), (13, None)):
        args = list(good)
        args[i] = bad
        assert LIB.tok_scan_grad(*args) == EINVAL, (i, bad)
    for i, bad in ((15, None), (15, p + 8), (16, nbytes - 1)):
        args = list(good)
        args[i] = bad
        assert LIB.tok_scan_grad(*args) == EWORKSPACE, (i, bad)
