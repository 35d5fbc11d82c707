"""Calls of the losses that would read what is not there, refused by the
binding before anything is allocated or enqueued."""
import pytest
import torch

import lsd_radix_sort_gb300 as rs


def f(*shape):
    return torch.zeros(*shape)


def i(*shape):
    return torch.zeros(*shape, dtype=torch.int64)


def test_backward_calls_without_lse():
    with pytest.raises(ValueError, match="needs the forward call's lse"):
        rs.distill_loss_backward(None, f(4, 9), None, f(4, 2), i(4, 2))
    with pytest.raises(ValueError, match="needs the forward call's lse"):
        rs.policy_loss_backward(None, f(4, 9), None, i(4), f(4), f(4))


CALLS = {
    "distill_loss": lambda **kw: rs.distill_loss(f(4, 9), f(4, 2), i(4, 2), **kw),
    "distill_loss_grad": lambda **kw: rs.distill_loss_grad(f(4, 9), f(4, 2), i(4, 2), **kw),
    "distill_loss_backward": lambda **kw: rs.distill_loss_backward(None, f(4, 9), f(4), f(4, 2), i(4, 2), **kw),
    "policy_loss": lambda **kw: rs.policy_loss(f(4, 9), i(4), f(4), f(4), **kw),
    "policy_loss_grad": lambda **kw: rs.policy_loss_grad(f(4, 9), i(4), f(4), f(4), **kw),
    "policy_loss_backward": lambda **kw: rs.policy_loss_backward(None, f(4, 9), f(4), i(4), f(4), f(4), **kw),
    "balance_loss": lambda **kw: rs.balance_loss(f(4, 9), i(4, 2), **kw),
    "balance_loss_grad": lambda **kw: rs.balance_loss_grad(f(4, 9), i(4, 2), **kw),
    "balance_loss_backward": lambda **kw: rs.balance_loss_backward(
        None, f(4, 9), i(9).int(), i(1).int(), 2, **kw),
}


class OtherStream:
    device_index = 0
    cuda_stream = 0


@pytest.mark.parametrize("name", sorted(CALLS))
def test_tensors_of_a_device_that_is_not_current(monkeypatch, name):
    """Device indices are stubbed: the tensors say that they are on the second
    device while the first is current."""
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 1)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="current CUDA device, got cuda:1 while cuda:0"):
        CALLS[name]()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="the stream must be one of cuda:1"):
        CALLS[name](stream=OtherStream())


@pytest.mark.parametrize("make,name", [("distill_args", "rs_distill_loss"), ("policy_args", "rs_policy_loss")])
def test_wait_limits_and_status(make, name):
    """By the C ABI: a limit above 60 s, a status word that is not aligned."""
    import ctypes

    from lsd_radix_sort_gb300 import build
    from tests import test_loss_checks as checks
    build.build()
    call = getattr(rs.load_library(), name)
    for change in (dict(wait_timeout_ns=60_000_000_001), dict(status=checks.BASE + 2)):
        assert call(ctypes.byref(getattr(checks, make)(**change)), None) == rs.RS_ERR_INVALID
