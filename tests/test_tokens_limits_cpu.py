"""What the token operators refuse, and where their limits lie, without a GPU."""
import ctypes

import torch
import torch.autograd.forward_ad as forward_ad
import pytest
from torch.fx.experimental.proxy_tensor import make_fx

import sparse_spatial_hashing_amd as ssh
from sparse_spatial_hashing_amd import tokens

LIB = tokens._lib
EINVAL = -1


# name, and a call of one float tensor among the operator's arguments
ROWS, HEADS = torch.zeros((4, 8)), torch.zeros((4, 1, 8), dtype=torch.bfloat16)
IDS, PLACES, SLOPES = torch.zeros(4, dtype=torch.int32), torch.zeros((4, 1), dtype=torch.int32), torch.zeros(1)
LSE, CARRY = torch.zeros((4, 1)), torch.zeros((1, 8))
CALLS = {
    "embed": (ROWS, lambda t: ssh.embed(t, IDS)),
    "embed_grad": (ROWS, lambda t: ssh.embed_grad(t, IDS, 4)),
    "attend q": (HEADS, lambda t: ssh.attend(t, HEADS, HEADS)),
    "attend v": (HEADS, lambda t: ssh.attend(HEADS, HEADS, t)),
    "attend slopes": (SLOPES, lambda t: ssh.attend(HEADS, HEADS, HEADS, slopes=t, q_pos=PLACES,
                                                   k_pos=PLACES)),
    "attend_grad": (HEADS, lambda t: ssh.attend_grad(t, HEADS, HEADS, HEADS, HEADS, LSE)),
    "gated_scan": (ROWS, lambda t: ssh.gated_scan(ROWS, t)[0]),
    "gated_scan state": (CARRY, lambda t: ssh.gated_scan(ROWS, ROWS, state=t)[0]),
    "gated_scan_grad": (ROWS, lambda t: ssh.gated_scan_grad(t, ROWS, ROWS, CARRY)[0]),
}


@pytest.mark.parametrize("name", CALLS)
def test_forward_mode_is_refused(name):
    """A dual tensor's tangent would be lost without a word: the call refuses before any other check."""
    t, call = CALLS[name]
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(t, torch.ones_like(t))
        with pytest.raises(NotImplementedError, match="forward-mode"):
            call(dual)
        with pytest.raises(ValueError, match="GPU"):  # no tangent: the next check
            call(t)


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("how", [dict(), dict(pre_dispatch=True), dict(tracing_mode="fake"), "jit"])
def test_tracing_is_refused(name, how):
    """A trace would hold the outputs' allocation and no kernel."""
    t, call = CALLS[name]
    with pytest.raises(NotImplementedError, match="traced"):
        if how == "jit":
            torch.jit.trace(call, t)
        else:
            make_fx(call, **how)(t)


def test_recurrence_steps_stay_in_32_bits():
    """The longest t accepted keeps the end of its last chunk (1024 steps at most) under 2^31."""
    most, p = 2**31 - 2048, 4096
    assert -(-most // 1024) * 1024 < 2**31
    assert LIB.tok_scan_runs(most) == most // tokens.TOK_SCAN_RUN
    nbytes = LIB.tok_scan_workspace_bytes(most, 1)
    assert nbytes > 0
    for t in (most + 1, 2**31 - 1024, 2**31 - 1):
        assert LIB.tok_scan_runs(t) == EINVAL and LIB.tok_scan_workspace_bytes(t, 1) == EINVAL
        assert LIB.tok_scan(p, p, 1, t, 1, p, 2, 0, p, p, p, p, p, 1 << 40, None) == EINVAL
        assert LIB.tok_scan_grad(p, p, p, p, 1, t, 1, p, 2, 0, p, p, p, p, p, p, 1 << 40, None) == EINVAL


def _attention(**more):
    base = dict(dtype=1, heads=1, kv_heads=1, width=8, tq=8, tk=8, docs=1, mask=0, scale=1.0, cap=0.0,
                q_stride=(8, 8), k_stride=(8, 8), v_stride=(8, 8), g_stride=(8, 8))
    base.update(more)
    return ctypes.byref(tokens._Attention(**base))


def test_attention_rows_stay_in_32_bits():
    """The most rows and keys accepted keep the end of a tile (128 at most) under 2^31."""
    most, p = 2**31 - 2048, 4096
    for good in (dict(tq=most), dict(tk=most), dict(tq=most // 16, heads=16, q_stride=(128, 8))):
        assert LIB.tok_attend_workspace_bytes(_attention(**good)) >= 0
        assert LIB.tok_attend_grad_workspace_bytes(_attention(**good)) >= 0
    for bad in (dict(tq=most + 1), dict(tk=most + 1), dict(tq=2**31 - 1, mask=1), dict(tk=2**31 - 100),
                dict(tq=most // 16 + 1, heads=16, q_stride=(128, 8)),
                dict(tk=most // 2 + 1, heads=2, kv_heads=2, k_stride=(16, 8))):
        a = _attention(**bad)
        assert LIB.tok_attend_workspace_bytes(a) == EINVAL and LIB.tok_attend_grad_workspace_bytes(a) == EINVAL
        assert LIB.tok_attend(a, p, p, p, p, None, p, 1 << 60, None) == EINVAL
        assert LIB.tok_attend_grad(a, *[p] * 10, 1 << 60, None) == EINVAL


def test_attention_blocks_stay_in_31_bits():
    """A tile per document and key head, and one per 32 rows or keys, for as many as are accepted."""
    strides = dict(q_stride=(8192, 8), k_stride=(8192, 8), v_stride=(8192, 8), g_stride=(8192, 8))
    for docs, kv_heads, good in ((2**20, 1023, True), (2**20, 1024, False), (16382, 65536, True),
                                 (16383, 65536, False)):
        a = _attention(docs=docs, heads=kv_heads, kv_heads=kv_heads, tq=4, tk=4, q_offsets=16, k_offsets=16,
                       **strides)
        assert (LIB.tok_attend_workspace_bytes(a) >= 0) == good, (docs, kv_heads)
        assert not good or 2**26 + (docs + 2) * kv_heads < 2**31
        if not good:
            assert LIB.tok_attend(a, *[4096] * 4, None, 4096, 1 << 60, None) == EINVAL


@pytest.mark.parametrize("cap,good", [(0.0, True), (2.0**-126, True), (30.0, True), (2.0**127, True),
                                      (2.0**-127, False), (2.5e38, False), (-2.0**-126, False)])
def test_attention_cap_limits(cap, good):
    a = _attention(cap=cap)
    assert (LIB.tok_attend_workspace_bytes(a) >= 0) == good
    assert (LIB.tok_attend_grad_workspace_bytes(a) >= 0) == good
