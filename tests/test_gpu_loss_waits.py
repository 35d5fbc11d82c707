"""The limit on the waits of the long rows' kernel: with one so short that
waits give up in the middle of their work, every row is either right or NaN
throughout, nothing is left of what the outputs held before, the status says
so, and the next call is right."""
import pytest
import torch

from tests.test_gpu_loss_order import Load

pytestmark = pytest.mark.gpu

# in the ring one CTA per row, more rows than SMs; clusters, one row each;
# clusters that take over further rows; rows of several rings
SHAPES = [(700, 40000, torch.bfloat16), (12, 40000, torch.bfloat16), (90, 200000, torch.float32),
          (400, 131072, torch.bfloat16), (170, 200003, torch.float32)]
LIMITS = [1, 300, 1000, 3000, 10000, 100000]


def check(got, want, status, rows):
    """got: losses, ..., gradient; want: the same of a call without a limit."""
    lost = got[0].isnan()
    for a, b in zip(got, want):
        a2, b2 = a.reshape(rows, -1), b.reshape(rows, -1)
        assert bool(a2[lost].isnan().all()), "a row is NaN in part"
        assert torch.equal(a2[~lost], b2[~lost]), "a row is wrong"
    if bool(lost.any()):
        assert int(status) == 4
    assert int(status) in (0, 4)
    return int(lost.sum())


@pytest.mark.parametrize("rows,cols,dtype", SHAPES)
def test_waits_that_give_up(rs, rows, cols, dtype):
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = (torch.randn(rows, cols, generator=g, device="cuda") * 3).to(dtype)
    values, indices = torch.topk(x, 12, dim=1)
    weights = torch.rand(rows, generator=g, device="cuda") + 0.5
    weights[torch.randperm(rows, generator=g, device="cuda")[:rows // 8]] = 0.0
    actions = indices[:, 3].contiguous()
    old = torch.log_softmax(x.float(), 1).gather(1, actions[:, None])[:, 0] + 0.05
    adv = torch.randn(rows, generator=g, device="cuda")
    grad = torch.empty_like(x)
    losses, logprobs, lse = (torch.empty(rows, device="cuda") for _ in range(3))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want_d = rs.distill_loss_grad(x, values, indices, weights=weights)
    want_p = rs.policy_loss_grad(x, actions, old, adv, weights=weights)
    lost = 0
    load = Load()  # copies take longer beside others
    for limit in LIMITS:
        for _ in range(3):
            load.more()
            for t in (grad, losses, logprobs, lse):
                t.fill_(12345.0)
            status.zero_()
            got = rs.distill_loss_grad(x, values, indices, weights=weights, losses_out=losses, lse_out=lse,
                                       grad_out=grad, wait_timeout_ns=limit, status_out=status)
            lost += check(got, want_d, status, rows)
            for t in (grad, losses, logprobs, lse):
                t.fill_(12345.0)
            status.zero_()
            got = rs.policy_loss_grad(x, actions, old, adv, weights=weights, losses_out=losses,
                                      logprobs_out=logprobs, lse_out=lse, grad_out=grad,
                                      wait_timeout_ns=limit, status_out=status)
            lost += check(got, want_p, status, rows)
    # with few rows the waits may all be met at once
    assert lost > 0 or rows == 12, "no wait gave up"
    status.zero_()
    again = rs.distill_loss_grad(x, values, indices, weights=weights, status_out=status)
    assert check(again, want_d, status, rows) == 0 and int(status) == 0


def test_limits_that_are_refused(rs):
    x = torch.zeros(4, 40000, device="cuda")
    v, i = torch.zeros(4, 2, device="cuda"), torch.zeros(4, 2, dtype=torch.int64, device="cuda")
    with pytest.raises(rs.RadixSortError):
        rs.distill_loss_grad(x, v, i, wait_timeout_ns=61_000_000_000)
    with pytest.raises(ValueError, match="status_out"):
        rs.distill_loss_grad(x, v, i, status_out=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="status_out"):
        rs.distill_loss_grad(x, v, i, status_out=torch.zeros(1, device="cuda"))
