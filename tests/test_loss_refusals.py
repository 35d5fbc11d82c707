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
