"""The 64-bit losses that the kernels are compared with: their gradients are
those of their losses (central differences, and torch's autograd over the
formulas), and their bounds notice planted mistakes."""
import math

import pytest
import torch

from tests import loss_oracle as lo


def case(rows=3, cols=11, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(rows, cols, generator=g, dtype=torch.float64) * 2, g


def differences(f, x, h=1e-6):
    out = torch.zeros_like(x)
    for i in range(x.shape[0]):
        for j in range(x.shape[1]):
            d = torch.zeros_like(x)
            d[i, j] = h
            out[i, j] = (f(x + d) - f(x - d)) / (2 * h)
    return out


@pytest.mark.parametrize("tau", [1.0, 0.7, 2.0])
def test_distill_gradient_is_the_losses(tau):
    x, g = case()
    values = torch.randn(3, 4, generator=g)
    indices = torch.tensor([[0, 5, 10, 3], [2, 2, 7, -1], [1, 11, 4, 4]])  # twice, dropped, outside
    w = torch.tensor([1.0, 0.5, -2.0])
    grad = lo.distill(x, values, indices, tau, w)[2]
    want = differences(lambda y: lo.distill(y, values, indices, tau, w)[0].sum(), x)
    assert torch.allclose(grad, want, atol=1e-8)  # h^2 and 1e-16 / h


def test_policy_gradient_is_the_losses():
    x, g = case(6)
    actions = torch.tensor([0, 3, 10, 5, 5, 2])
    logp = torch.log_softmax(x / 0.9, 1).gather(1, actions[:, None])[:, 0]
    old = logp + torch.tensor([0.0, 0.05, -0.5, 0.5, -0.5, 0.5])  # inside, and held both ways
    adv = torch.tensor([1.0, -1.0, 1.0, 1.0, -1.0, -1.0])
    ref = logp + 0.3
    kw = dict(ref=ref, low=0.1, high=0.3, kl=0.2, tau=0.9)
    grad = lo.policy(x, actions, old, adv, **kw)[3]
    want = differences(lambda y: lo.policy(y, actions, old, adv, **kw)[0].sum(), x)
    assert torch.allclose(grad, want, atol=1e-8)


def test_balance_gradient_is_the_losses():
    x, g = case(7, 5)
    ids = torch.tensor([[0, 1], [1, 2], [1, 4], [4, -1], [0, 0], [2, 5], [1, 3]])
    mask = torch.tensor([1, 1, 0, 1, 1, 1, 1], dtype=torch.bool)
    grad = lo.balance(x, ids, mask, 3.0)[4]
    want = differences(lambda y: torch.tensor(3.0 * lo.balance(y, ids, mask)[0], dtype=torch.float64), x)
    assert torch.allclose(grad, want, atol=1e-8)


def test_closed_forms():
    # a uniform row against a single certain target: log(cols)
    losses, lse, grad, _ = lo.distill(torch.zeros(1, 8), torch.zeros(1, 1), torch.tensor([[3]]))
    assert math.isclose(losses[0], math.log(8)) and math.isclose(lse[0], math.log(8))
    assert math.isclose(grad[0, 3], 1 / 8 - 1) and math.isclose(grad[0, 0], 1 / 8)
    # balanced experts: loss 1, gradient 0
    ids = torch.arange(8).reshape(4, 2) % 4
    loss, counts, mean, n, grad, _ = lo.balance(torch.zeros(4, 4), ids)
    assert math.isclose(loss, 1.0) and counts.tolist() == [2, 2, 2, 2] and n == 4
    assert float(grad.abs().max()) < 1e-15
    # ratio 1, no KL: loss -A
    x = torch.zeros(1, 4)
    out = lo.policy(x, torch.tensor([1]), torch.tensor([-math.log(4)], dtype=torch.float64),
                    torch.tensor([2.5]))
    assert math.isclose(out[0][0], -2.5)


def test_empty_rows_and_dropped_entries():
    x = torch.full((2, 5), -math.inf)
    x[1, 2] = 0.0
    losses, lse, grad, _ = lo.distill(x, torch.zeros(2, 2), torch.tensor([[0, 1], [2, -1]]))
    assert losses.tolist() == [0.0, 0.0] and lse[0] == -math.inf and lse[1] == 0.0
    assert float(grad.abs().max()) == 0.0
    out = lo.policy(x, torch.tensor([0, 9]), torch.zeros(2), torch.ones(2))
    assert out[0].tolist() == [0.0, 0.0] and out[1].tolist() == [-math.inf, 0.0]


def test_bounds_notice_mistakes():
    """A gradient without its targets, with a target's mass doubled, or with
    the temperature forgotten is outside the bounds that the kernels get."""
    g = torch.Generator().manual_seed(3)
    x = (torch.randn(2, 1000, generator=g) * 3).to(torch.bfloat16)
    values, indices = torch.topk(x.float() + torch.randn(2, 1000, generator=g), 8, dim=1)
    _, _, grad, size = lo.distill(x, values, indices, 2.0)
    bound = lo.grad_bound(grad, size, lo.row_error(x, 2.0), torch.bfloat16)
    lo.assert_within(grad.to(torch.bfloat16), grad, bound, "rounded")
    twice = torch.cat([indices, indices[:, :1]], 1), torch.cat([values, values[:, :1]], 1)
    for wrong in (lo.distill(x, values, torch.full_like(indices, -1), 2.0)[2],
                  lo.distill(x, twice[1], twice[0], 2.0)[2],
                  lo.distill(x, values, indices, 1.0)[2], grad * 1.02):
        with pytest.raises(AssertionError):
            lo.assert_within(wrong.to(torch.bfloat16), grad, bound, "mutant")
