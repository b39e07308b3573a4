"""What the operators' backward passes are given by torch, with the kernels' calls stood in for."""
import pytest
import torch

from sparse_spatial_hashing_amd import prediction


def _decay(monkeypatch, want_state=True):
    """decay_attend of three tokens under autograd, and the gradients that its backward is called with."""
    seen = []

    def forward(q, k, v, decay, offsets, state, scale, reverse, want_state):
        last = torch.ones((1, 1, 8, 8)) if want_state else None
        return q + k + v, last, torch.ones((2, 1, 8, 8))

    def backward(grad, q, k, v, decay, carry, offsets, state=None, grad_state=None, **how):
        seen.append((grad, grad_state))
        return grad, grad, grad, None if state is None else torch.full_like(state, 7.0)

    monkeypatch.setattr(prediction, "_decay_attend", forward)
    monkeypatch.setattr(prediction, "decay_attend_grad", backward)
    leaves = [torch.ones((3, 1, 8)).requires_grad_() for _ in range(3)] + [torch.ones((1, 1, 8, 8)).requires_grad_()]
    out, last, carry = prediction.decay_attend(*leaves[:3], torch.zeros(1), state=leaves[3], return_state=want_state,
                                               return_carry=True)
    assert not carry.requires_grad
    return leaves, out, last, seen


@pytest.mark.parametrize("want_state", [False, True])
def test_an_unused_state_has_no_gradient(monkeypatch, want_state):
    leaves, out, last, seen = _decay(monkeypatch, want_state)
    made = torch.autograd.grad(out.sum(), leaves)
    ((grad, grad_state),) = seen
    assert grad_state is None and torch.equal(grad, torch.ones_like(out))
    assert (made[3] == 7).all()


def test_an_unused_output_has_zeros(monkeypatch):
    leaves, out, last, seen = _decay(monkeypatch)
    made = torch.autograd.grad(last.sum(), leaves)
    ((grad, grad_state),) = seen
    assert grad.shape == out.shape and not grad.any() and torch.equal(grad_state, torch.ones_like(last))
    assert not made[0].any() and (made[3] == 7).all()


def test_both_outputs(monkeypatch):
    leaves, out, last, seen = _decay(monkeypatch)
    torch.autograd.grad((out, last), leaves, (2 * torch.ones_like(out), 3 * torch.ones_like(last)))
    ((grad, grad_state),) = seen
    assert (grad == 2).all() and (grad_state == 3).all()


def test_the_sum_of_the_weights_has_no_gradient(monkeypatch):
    """row_loss's second output is not differentiable: no zeros are made for it."""
    seen = []
    monkeypatch.setattr(prediction, "_row_loss", lambda x, table, ids, scale, want: (x.sum(1), x.sum(1)))
    monkeypatch.setattr(prediction, "_row_loss_grad", lambda *a: seen.append(a) or (a[1], a[2]))
    zeros = []
    plain = prediction._RowLoss.backward

    def backward(ctx, grad, grad_lse):
        zeros.append(grad_lse)
        return plain(ctx, grad, grad_lse)

    monkeypatch.setattr(prediction._RowLoss, "backward", staticmethod(backward))
    leaves = [torch.ones((4, 8)).requires_grad_(), torch.ones((5, 8)).requires_grad_()]
    loss, lse = prediction.row_loss(*leaves, torch.zeros(4, dtype=torch.int64), return_lse=True)
    assert not lse.requires_grad
    torch.autograd.grad(loss.sum(), leaves)
    assert zeros == [None] and torch.equal(seen[0][0], torch.ones(4))
