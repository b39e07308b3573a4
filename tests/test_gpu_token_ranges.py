"""Token operators on the GPU where the elements' type is narrow: values far
below and above 1, against the 64-bit definitions. Bounds are those of
token_reference with half a step of the type's smallest numbers instead of its
smallest normal number."""
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


def _ends(lens):
    return [0] + torch.tensor(lens).cumsum(0).tolist()


def _at(ends):
    return torch.tensor(ends, dtype=torch.int32, device=DEV)


def _check(got, want, dtype, what):
    """As ref.check, but results under the smallest normal number count too."""
    tiny = torch.finfo(dtype).smallest_normal
    ref.check(got, want[0], want[1] - tiny + tiny * ref.unit(dtype), what)


def _gradients(q, k, v, grad, ends, what, **more):
    scale = q.shape[2] ** -0.5
    want = ref.attend(q, k, v, ends, ends, scale, grad=grad, **more)
    print(what, flush=True)
    m = dict({n: x.to(DEV) if isinstance(x, torch.Tensor) else x for n, x in more.items()},
             q_offsets=_at(ends), k_offsets=_at(ends))
    q, k, v, grad = (t.to(DEV) for t in (q, k, v, grad))
    out, lse = ssh.attend(q, k, v, return_lse=True, **m)
    return dict(zip(("gq", "gk", "gv"), ssh.attend_grad(grad, q, k, v, out, lse, **m))), want


SIZES = [([2000], 64, 0, 0.0, False), ([40, 33, 7], 32, 3, 20.0, False), ([900, 300], 128, 2, 0.0, True),
         ([60, 2], 128, 0, 30.0, True)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("size", [1e-6, 1e-3, 1e4])
@pytest.mark.parametrize("lens,width,axes,cap,causal", SIZES)
def test_gradients_of_any_size(dtype, size, lens, width, axes, cap, causal):
    """Score gradients far under the type's smallest number, and over its largest. Large keys
    bring grad_q back into range, large queries grad_k."""
    gen = torch.Generator().manual_seed(width)
    ends, heads = _ends(lens), 2
    n = ends[-1]
    more = dict(cap=cap, causal=causal)
    if axes:
        pos = (torch.rand((n, axes), generator=gen) * 40).int()
        more.update(q_pos=pos, k_pos=pos, slopes=torch.tensor([0.125, 0.03125]))
    grow = torch.exp2(torch.linspace(-6, 3, n))[:, None, None]  # along the tokens: later ones count most
    for by, back in (("gq", False), ("gk", False), ("gq", True), ("gk", True)):
        large, little = (50.0, 0.02) if size < 1 else (0.02, 0.02)
        std = dict(gq=(little, large), gk=(large, little))[by]
        q, k = (torch.randn((n, h, width), generator=gen) * s for h, s in zip((heads, 1), std))
        v, grad = torch.randn((n, 1, width), generator=gen), torch.randn((n, heads, width), generator=gen)
        v, grad = v * (grow.flip(0) if back else grow), grad * size / grow.max() * (grow if back else 1.0)
        q, k, v, grad = (t.to(dtype) for t in (q, k, v, grad))
        made, want = _gradients(q, k, v, grad, ends, f"{by} of size {size} {lens} w {width} {dtype}", **more)
        _check(made[by], want[by], dtype, f"{by} of size {size} {lens} w {width} {dtype}")


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("lens,width", [([70], 64), ([30, 300], 128), ([500], 32)])
def test_gradients_through_small_weights(dtype, lens, width):
    """Keys of weights down to e^-16 and large gradients: grad_v keeps them."""
    gen = torch.Generator().manual_seed(width)
    ends = _ends(lens)
    n = ends[-1]
    q, k, v, grad = (torch.randn((n, 1, width), generator=gen) for _ in range(4))
    q[..., 0], k[..., 0] = 4.0, torch.linspace(0, -16, n)[:, None] * width ** 0.5 / 4
    made, want = _gradients(q.to(dtype), k.to(dtype), v.to(dtype), (grad * 500).to(dtype), ends,
                            f"small weights {lens} w {width} {dtype}")
    for name in ("gq", "gk", "gv"):
        _check(made[name], want[name], dtype, f"{name} small weights {lens} w {width} {dtype}")


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("q_len,width,place,axes", [(1, 128, 0, 0), (1, 64, 0, 2), (40, 32, 0, 0), (150, 64, 0, 3),
                                                    (150, 128, 0, 0), (70, 128, 5000, 2), (1, 80, 19999, 0)])
def test_many_small_weights(dtype, q_len, width, place, axes):
    """One key with nearly all the weight and a value of zero: the output is what 20,000 keys of
    e^-17.5 its weight add up to."""
    gen = torch.Generator().manual_seed(width)
    n = 20000
    q, k, v = (torch.randn((m, 1, width), generator=gen) * s for m, s in ((q_len, 0.1), (n, 0.1), (n, 0.1)))
    q[..., 0], k[..., 0], k[place, 0, 0] = 4.0, 0.0, 17.5 * width ** 0.5 / 4
    v += 1.0
    v[place] = 0.0
    q, k, v = (t.to(dtype) for t in (q, k, v))
    more = {}
    if axes:
        more = dict(q_pos=torch.ones((q_len, axes), dtype=torch.int32),
                    k_pos=torch.ones((n, axes), dtype=torch.int32), slopes=torch.tensor([0.5]))
    want = ref.attend(q, k, v, [0, q_len], [0, n], width ** -0.5, **more)
    what = f"small weights {q_len} w {width} at {place} {dtype}"
    print(what, flush=True)
    more = {name: t.to(DEV) for name, t in more.items()}
    out, lse = ssh.attend(q.to(DEV), k.to(DEV), v.to(DEV), return_lse=True, **more)
    _check(out, want["out"], dtype, what)
    ref.check(lse, *want["lse"], what + " lse")


def test_forward_mode_and_traces_are_refused_and_compilation_goes_round():
    """torch sees no kernel: what would lose them raises, torch.compile leaves the call as it is."""
    import torch.autograd.forward_ad as forward_ad
    from torch.fx.experimental.proxy_tensor import make_fx
    gen = torch.Generator().manual_seed(1)
    table = torch.randn((9, 8), generator=gen).to(DEV)
    ids = torch.randint(0, 9, (40,), generator=gen).to(DEV)
    h = torch.randn((40, 2, 16), generator=gen).to(DEV, BF16)
    calls = ((table, lambda t: ssh.embed(t, ids)), (h, lambda t: ssh.attend(t, h, h)),
             (table, lambda t: ssh.gated_scan(t, table)[0]))
    for t, call in calls:
        with forward_ad.dual_level(), pytest.raises(NotImplementedError):
            call(forward_ad.make_dual(t, torch.ones_like(t)))
        with forward_ad.dual_level(), pytest.raises(NotImplementedError):
            call(forward_ad.make_dual(t.clone().requires_grad_(), torch.ones_like(t)))
        with pytest.raises(NotImplementedError):
            make_fx(call)(t)
        torch._dynamo.reset()
        assert torch.equal(torch.compile(lambda x: call(x) * 2, backend="eager")(t), call(t) * 2)


def test_embed_more_rows_than_one_launch_holds():
    """67 M rows of 129, four to a block: 2^24 blocks of 256 threads, one more than a launch takes."""
    n, width = (1 << 26) + 5, 129
    gen = torch.Generator().manual_seed(4)
    table = torch.randn((50, width), generator=gen).to(DEV, F16)
    ids = (torch.arange(n, device=DEV, dtype=torch.int32) * 7) % 53 - 2
    print(f"embed {n} rows of {width}", flush=True)
    out = ssh.embed(table, ids)
    where = torch.cat([torch.arange(2000), torch.arange((1 << 26) - 2000, n),
                       torch.randint(0, n, (100000,), generator=gen)]).to(DEV)
    i = ids[where].long()
    want = torch.where((i >= 0)[:, None] & (i < 50)[:, None], table[i.clamp(0, 49)], 0)
    assert torch.equal(out[where], want)


def test_attend_more_blocks_than_one_launch_holds():
    """A million sequences of one token, 64 heads: 69 M blocks of a wavefront, 2^26 and more. The one
    key's weight is 1, so the output is its value."""
    n, heads, width = 1 << 20, 64, 8
    at = torch.arange(n + 1, dtype=torch.int32, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(5)
    q, k, v, grad = (torch.randn((n, heads, width), generator=gen, device=DEV, dtype=BF16) for _ in range(4))
    print(f"attend {n} documents, {heads} heads", flush=True)
    out, lse = ssh.attend(q, k, v, q_offsets=at, k_offsets=at, return_lse=True)
    assert torch.equal(out, v)
    want = (q.float() * k.float()).sum(2) * width ** -0.5
    assert ((lse - want).abs() <= 2.0 ** -18 * (1 + (q.float() * k.float()).abs().sum(2))).all()
    gq, gk, gv = ssh.attend_grad(grad, q, k, v, out, lse, q_offsets=at, k_offsets=at)
    assert torch.equal(gv, grad) and not gq.any() and not gk.any()


def _odd(tokens, heads, width, of=13):
    """A view whose strides are not whole 16-byte pieces."""
    return torch.ones((tokens, heads, of), dtype=BF16, device=DEV)[..., 3:3 + width]


@pytest.mark.parametrize("tq,tk", [(0, 0), (0, 5), (5, 0)])
def test_attend_nothing_in_odd_strides(tq, tk):
    """A layout that is copied where there are tokens does where there are none."""
    leaves = [t.detach().requires_grad_() for t in (_odd(tq, 2, 8), _odd(tk, 1, 8), _odd(tk, 1, 8, 15))]
    out, lse = ssh.attend(*leaves, return_lse=True)
    assert out.shape == (tq, 2, 8) and not out.any() and torch.isneginf(lse).all()
    for grad in (_odd(tq, 2, 8, 11), torch.ones((), dtype=BF16, device=DEV).expand(tq, 2, 8)):
        made = torch.autograd.grad(out, leaves, grad, retain_graph=True)
        assert all(g.shape == t.shape and not g.any() for g, t in zip(made, leaves))
    at = torch.zeros(3, dtype=torch.int32, device=DEV)
    with torch.no_grad():
        assert not ssh.attend(*leaves, q_offsets=at, k_offsets=at).any()
        assert not ssh.attend(leaves[0][3:], leaves[1][3:], leaves[2][3:]).any()


@pytest.mark.parametrize("rows,n", [((1 << 24) + 1, 3), (3, (1 << 27) + 1)])
def test_embed_refuses_a_gradient_it_cannot_give(rows, n):
    """Before the forward, not in the backward; without a gradient the same lookup runs."""
    table = torch.ones((rows, 1), device=DEV, dtype=F16)
    ids = torch.full((n,), rows - 1, dtype=torch.int32, device=DEV)
    assert ssh.embed(table, ids).all()
    with pytest.raises(ValueError, match="gradient"):
        ssh.embed(table.requires_grad_(), ids)
    with torch.no_grad():
        assert ssh.embed(table, ids).all()
    less = table.detach()[:1 << 24].requires_grad_()
    assert ssh.embed(less, ids[:1000]).requires_grad


def test_attend_learned_slopes_without_gradients():
    """Slopes of a parameter serve where gradients are off; elsewhere theirs would be lost."""
    gen = torch.Generator().manual_seed(6)
    q, k = (torch.randn((30, h, 32), generator=gen).to(DEV, BF16) for h in (4, 2))
    pos = torch.randint(0, 50, (30, 2), generator=gen, dtype=torch.int32).to(DEV)
    slopes = torch.tensor([0.5, 0.25, 0.1, 0.0], device=DEV)
    learned = slopes.clone().requires_grad_()
    m = dict(q_pos=pos, k_pos=pos)
    want, lse = ssh.attend(q, k, k, slopes=slopes, return_lse=True, **m)
    for off in (torch.no_grad(), torch.inference_mode()):
        with off:
            assert torch.equal(ssh.attend(q, k, k, slopes=learned, **m), want)
            ssh.attend_grad(q, q, k, k, want, lse, slopes=learned, **m)
    for call in (lambda: ssh.attend(q, k, k, slopes=learned, **m),
                 lambda: ssh.attend(q.clone().requires_grad_(), k, k, slopes=learned, **m),
                 lambda: ssh.attend_grad(q, q, k, k, want, lse, slopes=learned, **m)):
        with pytest.raises(ValueError, match="slopes"):
            call()


@pytest.mark.parametrize("cap,scale", [(2.0**-126, 1.0), (1e-30, 1e30), (2.0**127, 0.25), (1e30, 0.25)])
def test_attend_extreme_caps(cap, scale):
    """A cap so small that scale / cap passes the floats (scores of exactly 0 among them), and one so
    large that it bends nothing."""
    gen = torch.Generator().manual_seed(8)
    q, k, v, grad = (torch.randn((50, 1, 32), generator=gen).to(BF16) for _ in range(4))
    q[3], k[7] = 0.0, 0.0
    want = ref.attend(q, k, v, [0, 50], [0, 50], scale, cap=cap, grad=grad)
    m = dict(cap=cap, scale=scale)
    g = [t.to(DEV) for t in (q, k, v, grad)]
    out, lse = ssh.attend(*g[:3], return_lse=True, **m)
    ref.check(out, *want["out"], f"out cap {cap}")
    ref.check(lse, *want["lse"], f"lse cap {cap}")
    made = ssh.attend_grad(g[3], *g[:3], out, lse, **m)
    for name, t in zip(("gq", "gk", "gv"), made):
        if name == "gv" or cap > 1:  # bent flat: the formula's 64 bits leave 1e-30 of a gradient of 1e30
            ref.check(t, *want[name], f"{name} cap {cap}")
        else:
            assert torch.isfinite(t).all()


@pytest.mark.parametrize("cap", [1e-50, 2.0**-127, 2.5e38, 1e39, math.inf, math.nan, -1e-50])
def test_attend_refuses_caps(cap):
    h = torch.zeros((4, 2, 16), device=DEV, dtype=BF16)
    with pytest.raises(ValueError):
        ssh.attend(h, h, h, cap=cap)
