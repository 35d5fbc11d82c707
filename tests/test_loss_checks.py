"""What the losses over rows of scores refuse, before anything is enqueued: by
the binding (types, shapes, strides, devices) and by the C ABI itself."""
import ctypes

import pytest
import torch

import lsd_radix_sort_gb300 as rs
from lsd_radix_sort_gb300 import losses


@pytest.fixture(scope="module")
def lib():
    from lsd_radix_sort_gb300 import build
    build.build()
    return rs.load_library()


def f(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


def i(*shape, dtype=torch.int64):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("error,match,call", [
    (TypeError, "float16, bfloat16 or float32", lambda: rs.distill_loss(f(4, 9, dtype=torch.float64), f(4, 2), i(4, 2))),
    (TypeError, "top_values", lambda: rs.distill_loss(f(4, 9), i(4, 2), i(4, 2))),
    (TypeError, "int32 or int64", lambda: rs.distill_loss(f(4, 9), f(4, 2), i(4, 2, dtype=torch.int16))),
    (ValueError, "2-D", lambda: rs.distill_loss(f(9), f(4, 2), i(4, 2))),
    (ValueError, "both have shape", lambda: rs.distill_loss(f(4, 9), f(4, 2), i(4, 3))),
    (ValueError, "both have shape", lambda: rs.distill_loss(f(4, 9), f(3, 2), i(3, 2))),
    (ValueError, "top logits per row", lambda: rs.distill_loss(f(4, 9), f(4, 0), i(4, 0))),
    (ValueError, "top logits per row", lambda: rs.distill_loss(f(4, 9), f(4, 1025), i(4, 1025))),
    (ValueError, "unit stride", lambda: rs.distill_loss(f(9, 4).t(), f(4, 2), i(4, 2))),
    (ValueError, "unit stride", lambda: rs.distill_loss(f(4, 9), f(4, 2), i(2, 4).t())),
    (ValueError, "do not overlap", lambda: rs.distill_loss(f(1, 9).expand(4, 9), f(4, 2), i(4, 2))),
    (ValueError, "weights", lambda: rs.distill_loss(f(4, 9), f(4, 2), i(4, 2), weights=f(3))),
    (ValueError, "weights", lambda: rs.distill_loss(f(4, 9), f(4, 2), i(4, 2), weights=f(4, dtype=torch.float16))),
    (ValueError, "weights must be contiguous", lambda: rs.distill_loss(f(4, 9), f(4, 2), i(4, 2), weights=f(8)[::2])),
    (ValueError, "losses_out", lambda: rs.distill_loss(f(4, 9), f(4, 2), i(4, 2), losses_out=f(5))),
    (ValueError, "grad_out", lambda: rs.distill_loss_grad(f(4, 9), f(4, 2), i(4, 2), grad_out=f(4, 8))),
    (ValueError, "grad_out", lambda: rs.distill_loss_grad(f(4, 9), f(4, 2), i(4, 2), grad_out=f(4, 9, dtype=torch.float16))),
    (ValueError, "lse", lambda: rs.distill_loss_backward(None, f(4, 9), f(3), f(4, 2), i(4, 2))),
    (ValueError, "CUDA", lambda: rs.distill_loss(f(4, 9), f(4, 2), i(4, 2))),
    (TypeError, "actions", lambda: rs.policy_loss(f(4, 9), f(4), f(4), f(4))),
    (ValueError, "actions", lambda: rs.policy_loss(f(4, 9), i(5), f(4), f(4))),
    (ValueError, "old_logprobs", lambda: rs.policy_loss(f(4, 9), i(4), f(3), f(4))),
    (ValueError, "advantages", lambda: rs.policy_loss(f(4, 9), i(4), f(4), f(4, dtype=torch.float64))),
    (ValueError, "needs ref_logprobs", lambda: rs.policy_loss(f(4, 9), i(4), f(4), f(4), kl_coef=0.1)),
    (ValueError, "CUDA", lambda: rs.policy_loss(f(4, 9), i(4), f(4), f(4))),
    (ValueError, "shape", lambda: rs.balance_loss(f(4, 9), i(3, 2))),
    (ValueError, "shape", lambda: rs.balance_loss(f(4, 9), i(4))),
    (ValueError, "experts", lambda: rs.balance_loss(f(4, 1025), i(4, 2))),
    (ValueError, "token_mask", lambda: rs.balance_loss(f(4, 9), i(4, 2), token_mask=f(4))),
    (ValueError, "token_mask", lambda: rs.balance_loss(f(4, 9), i(4, 2), token_mask=torch.ones(3, dtype=torch.bool))),
    (ValueError, "CUDA", lambda: rs.balance_loss(f(4, 9), i(4, 2))),
    (ValueError, "counts", lambda: rs.balance_loss_backward(f(1), f(4, 9), i(9), i(1, dtype=torch.int32), 2)),
    (ValueError, "n_tokens", lambda: rs.balance_loss_backward(f(1), f(4, 9), i(9, dtype=torch.int32), i(2, dtype=torch.int32), 2)),
    (ValueError, "one float32", lambda: rs.balance_loss_backward(f(2), f(4, 9), i(9, dtype=torch.int32), i(1, dtype=torch.int32), 2)),
    (ValueError, "top_k", lambda: rs.balance_loss_backward(f(1), f(4, 9), i(9, dtype=torch.int32), i(1, dtype=torch.int32), 0)),
])
def test_binding_refuses(error, match, call):
    with pytest.raises(error, match=match):
        call()


BASE = 0x10000000  # addresses that no call here may touch


def distill_args(**change):
    a = dict(logits=BASE, logits_stride=100, rows=4, cols=100, top_values=BASE + 0x100000,
             top_values_stride=8, top_indices=BASE + 0x200000, top_indices_stride=8, weights=None,
             losses=BASE + 0x300000, lse=BASE + 0x310000, grad=BASE + 0x400000, grad_stride=100,
             logits_type=1, top_values_type=1, index_bytes=8, top=8, temperature=1.0)
    return losses.DistillArgs(**{**a, **change})


def policy_args(**change):
    a = dict(logits=BASE, logits_stride=100, rows=4, cols=100, actions=BASE + 0x100000,
             old_logprobs=BASE + 0x110000, advantages=BASE + 0x120000, ref_logprobs=None,
             weights=None, losses=BASE + 0x300000, logprobs=BASE + 0x320000, lse=BASE + 0x310000,
             grad=BASE + 0x400000, grad_stride=100, logits_type=1, index_bytes=8, clip_low=0.2,
             clip_high=0.2, kl_coef=0.0, temperature=1.0)
    return losses.PolicyArgs(**{**a, **change})


def balance_args(**change):
    a = dict(scores=BASE, scores_stride=64, tokens=4, expert_ids=BASE + 0x100000,
             expert_ids_stride=2, token_mask=None, loss=BASE + 0x200000, mean_probs=BASE + 0x210000,
             counts=BASE + 0x220000, n_tokens=BASE + 0x230000, grad=BASE + 0x400000, grad_stride=64,
             temp=BASE + 0x500000, temp_bytes=1 << 30, scores_type=0, experts=64, index_bytes=8,
             top=2, scale=1.0)
    return losses.BalanceArgs(**{**a, **change})


NAN, INF = float("nan"), float("inf")
SHARED = [dict(logits_type=3), dict(logits_type=-1), dict(rows=-1), dict(rows=1 << 31),
          dict(cols=0), dict(cols=1 << 30), dict(logits_stride=99), dict(logits_stride=1 << 61),
          dict(temperature=0.0), dict(temperature=-1.0), dict(temperature=NAN),
          dict(temperature=INF), dict(temperature=1e-45), dict(logits=None), dict(logits=BASE + 1),
          dict(losses=None), dict(losses=BASE + 0x300002), dict(lse=None), dict(weights=BASE + 2),
          dict(grad_stride=99), dict(grad=BASE + 0x400001), dict(grad=BASE + 2),
          dict(grad=BASE, grad_stride=101), dict(index_bytes=2)]


@pytest.mark.parametrize("change", SHARED + [
    dict(top=0), dict(top=1025), dict(top_values_type=5), dict(top_values=None),
    dict(top_values=BASE + 0x100001), dict(top_indices=BASE + 0x200004), dict(top_indices=None),
    dict(top_values_stride=7), dict(top_indices_stride=7)])
def test_distill_refuses(lib, change):
    assert lib.rs_distill_loss(ctypes.byref(distill_args(**change)), None) == rs.RS_ERR_INVALID


@pytest.mark.parametrize("change", SHARED + [
    dict(actions=None), dict(actions=BASE + 0x100004), dict(old_logprobs=None),
    dict(advantages=None), dict(ref_logprobs=BASE + 1), dict(kl_coef=0.1), dict(kl_coef=NAN),
    dict(clip_low=-0.1), dict(clip_low=NAN), dict(clip_high=-0.1), dict(clip_high=INF),
    dict(logprobs=None)])
def test_policy_refuses(lib, change):
    assert lib.rs_policy_loss(ctypes.byref(policy_args(**change)), None) == rs.RS_ERR_INVALID


@pytest.mark.parametrize("change,status", [
    (dict(scores_type=3), 1), (dict(tokens=-1), 1), (dict(tokens=1 << 30, top=2), 1),
    (dict(experts=0), 1), (dict(experts=1025, scores_stride=1025), 1), (dict(scores_stride=63), 1),
    (dict(expert_ids_stride=1), 1), (dict(index_bytes=1), 1), (dict(top=0), 1),
    (dict(scores=None), 1), (dict(scores=BASE + 1), 1), (dict(expert_ids=None), 1),
    (dict(expert_ids=BASE + 0x100004), 1), (dict(loss=None), 1), (dict(mean_probs=None), 1),
    (dict(counts=None), 1), (dict(n_tokens=None), 1), (dict(grad_stride=63), 1),
    (dict(grad=BASE + 2), 1), (dict(scale=NAN), 1),
    (dict(tokens=1 << 20, grad=None, temp=None), 1),          # large calls need scratch
    (dict(tokens=1 << 20, grad=None, temp=BASE + 0x500010), 1),
    (dict(tokens=1 << 20, grad=None, temp_bytes=64), 2)])
def test_balance_refuses(lib, change, status):
    assert lib.rs_balance_loss(ctypes.byref(balance_args(**change)), None) == status


def test_backward_calls_refuse(lib):
    bad = ctypes.c_void_p(BASE + 2)
    assert lib.rs_distill_loss_backward(ctypes.byref(distill_args(grad=None)), None, None) == 1
    assert lib.rs_distill_loss_backward(ctypes.byref(distill_args(lse=None)), None, None) == 1
    assert lib.rs_distill_loss_backward(ctypes.byref(distill_args()), bad, None) == 1
    assert lib.rs_policy_loss_backward(ctypes.byref(policy_args(grad=None)), None, None) == 1
    assert lib.rs_policy_loss_backward(ctypes.byref(policy_args()), bad, None) == 1
    assert lib.rs_balance_loss_backward(ctypes.byref(balance_args(grad=None)), None, None) == 1
    assert lib.rs_balance_loss_backward(ctypes.byref(balance_args()), bad, None) == 1
    for name in ("distill", "policy", "balance"):
        assert getattr(lib, f"rs_{name}_loss")(None, None) == 1
        assert getattr(lib, f"rs_{name}_loss_backward")(None, None, None) == 1


def test_no_rows_is_no_work(lib):
    none = dict(logits=None, losses=None, lse=None, grad=None)
    assert lib.rs_distill_loss(ctypes.byref(distill_args(rows=0, top_values=None, top_indices=None, **none)), None) == 0
    assert lib.rs_policy_loss(ctypes.byref(policy_args(rows=0, **none)), None) == 0
    assert lib.rs_balance_loss_backward(ctypes.byref(balance_args(tokens=0, scores=None, grad=None)), None, None) == 0


def test_wait_probe_refuses(lib):
    out = ctypes.c_int(0)
    for word, limit in ((None, 1), (ctypes.c_void_p(BASE + 2), 1), (ctypes.c_void_p(BASE), 0),
                        (ctypes.c_void_p(BASE), 61_000_000_000)):
        assert lib.rs_row_wait_timeout_probe(word, limit, None, ctypes.byref(out)) == 1
    assert lib.rs_row_wait_timeout_probe(ctypes.c_void_p(BASE), 1, None, None) == 1


def test_balance_scratch_size(lib):
    out = ctypes.c_size_t(0)
    for bad in ((-1, 8), (10, 0), (10, 1025)):
        assert lib.rs_balance_temp_bytes(*bad, ctypes.byref(out)) == 1
    assert lib.rs_balance_temp_bytes(10, 8, None) == 1
    assert rs.balance_temp_bytes(10, 8) == 0
    assert rs.balance_temp_bytes(1 << 20, 1024) > rs.balance_temp_bytes(1 << 20, 8) > 0
