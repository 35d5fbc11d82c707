"""Losses over rows of scores: binding of the ``rs_*_loss`` entry points.

``distill_loss`` takes a student's rows of logits and the top values and
columns of its teacher's (what a descending ``segmented_sort`` returns, cut to
the first k), ``policy_loss`` rows of logits and one sampled column each, and
``balance_loss`` a router's rows of scores and the expert ids chosen in them.
Each comes in three forms:

  ``*_loss``           the losses (differentiable by torch's autograd with
                       respect to the scores when those require a gradient)
  ``*_loss_grad``      the losses and the gradient of their (weighted) sum, in
                       one read of the scores: what a training step that knows
                       its weights beforehand uses
  ``*_loss_backward``  the gradient for upstream gradients, from the
                       statistics that the first form returned

The formulas, and what happens to masked rows, dropped entries, -inf and NaN,
are stated in include/lsdrs.h.  As in the rest of the package the work is
enqueued on ``stream`` (the current stream by default) and nothing
synchronises; results are allocated by torch on that stream unless given.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import types

from . import _check, _lib_of

__all__ = [
    "distill_loss", "distill_loss_grad", "distill_loss_backward", "policy_loss",
    "policy_loss_grad", "policy_loss_backward", "balance_loss", "balance_loss_grad",
    "balance_loss_backward", "balance_temp_bytes", "row_wait_timeout_probe", "MAX_TOP",
    "MAX_EXPERTS",
]

MAX_TOP = 1024
MAX_EXPERTS = 1024

_P, _I64, _U64, _I, _F, _SZ = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint64, ctypes.c_int,
                               ctypes.c_float, ctypes.c_size_t)


class DistillArgs(ctypes.Structure):
    """struct rs_distill_args of include/lsdrs.h."""
    _fields_ = [("logits", _P), ("logits_stride", _I64), ("rows", _I64), ("cols", _I64),
                ("top_values", _P), ("top_values_stride", _I64), ("top_indices", _P),
                ("top_indices_stride", _I64), ("weights", _P), ("losses", _P), ("lse", _P),
                ("grad", _P), ("grad_stride", _I64), ("logits_type", _I),
                ("top_values_type", _I), ("index_bytes", _I), ("top", _I), ("temperature", _F),
                ("wait_timeout_ns", _U64), ("status", _P)]


class PolicyArgs(ctypes.Structure):
    """struct rs_policy_args of include/lsdrs.h."""
    _fields_ = [("logits", _P), ("logits_stride", _I64), ("rows", _I64), ("cols", _I64),
                ("actions", _P), ("old_logprobs", _P), ("advantages", _P), ("ref_logprobs", _P),
                ("weights", _P), ("losses", _P), ("logprobs", _P), ("lse", _P), ("grad", _P),
                ("grad_stride", _I64), ("logits_type", _I), ("index_bytes", _I),
                ("clip_low", _F), ("clip_high", _F), ("kl_coef", _F), ("temperature", _F),
                ("wait_timeout_ns", _U64), ("status", _P)]


class BalanceArgs(ctypes.Structure):
    """struct rs_balance_args of include/lsdrs.h."""
    _fields_ = [("scores", _P), ("scores_stride", _I64), ("tokens", _I64), ("expert_ids", _P),
                ("expert_ids_stride", _I64), ("token_mask", _P), ("loss", _P),
                ("mean_probs", _P), ("counts", _P), ("n_tokens", _P), ("grad", _P),
                ("grad_stride", _I64), ("temp", _P), ("temp_bytes", _SZ), ("scores_type", _I),
                ("experts", _I), ("index_bytes", _I), ("top", _I), ("scale", _F)]


# torch, its score types and its raw current stream, once a call has needed them
_torch = None
_TYPES = {}
_raw_stream = None


def _load():
    global _torch, _raw_stream
    import torch
    _TYPES.update({torch.float16: 0, torch.bfloat16: 1, torch.float32: 2})
    # the current stream's address without a Stream object around it, where
    # this torch has that call
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda index: torch.cuda.current_stream(index).cuda_stream)
    _torch = torch
    return torch


def _kind(t, what):
    """The rs_score_type of a tensor of scores."""
    kind = _TYPES.get(t.dtype)
    if kind is None:
        raise TypeError(f"{what} must be float16, bfloat16 or float32, got {t.dtype}")
    return kind


def _matrix(t, what):
    """(rows, cols, elements from one row to the next) of a 2-D tensor with unit
    stride in its rows (a lone row's stride means nothing)."""
    if t.dim() != 2:
        raise ValueError(f"{what} must be a 2-D tensor")
    rows, cols = t.shape
    stride, unit = t.stride()
    if unit != 1 and cols > 1:
        raise ValueError(f"{what} must have unit stride in its last dimension")
    if rows <= 1:
        return rows, cols, cols
    if stride < cols:
        raise ValueError(f"{what} must have rows that do not overlap")
    return rows, cols, stride


def _index_bytes(t, what):
    if t.dtype is _torch.int64:
        return 8
    if t.dtype is _torch.int32:
        return 4
    raise TypeError(f"{what} must be int32 or int64, got {t.dtype}")


def _vector(t, n, what, dtype=None):
    """A contiguous vector of n elements (float32 unless dtype is given)."""
    if t.dtype is not (_torch.float32 if dtype is None else dtype) or t.shape != (n,):
        raise ValueError(f"{what} must be {dtype or _torch.float32} of shape ({n},), got "
                         f"{t.dtype} of {tuple(t.shape)}")
    if n > 1 and t.stride(0) != 1:
        raise ValueError(f"{what} must be contiguous")


def _device(stream, x, *ts):
    """The index of the one CUDA device that all tensors are on, which must be
    the current one (the library launches there) and the stream's."""
    index = x.get_device()
    if index < 0:
        raise ValueError("tensors must be on a CUDA device")
    for t in ts:
        if t is not None and t.get_device() != index:
            raise ValueError("tensors must be on one CUDA device")
    if index != _torch.cuda.current_device():
        raise ValueError(f"tensors must be on the current CUDA device, got cuda:{index} while "
                         f"cuda:{_torch.cuda.current_device()} is current")
    if stream is not None and stream.device_index != index:
        raise ValueError(f"the stream must be one of cuda:{index}, the tensors' device")
    return index


def _grad_stride(x, grad_out):
    if grad_out.dtype is not x.dtype or grad_out.shape != x.shape:
        raise ValueError(f"grad_out must be {x.dtype} of shape {tuple(x.shape)}")
    return _matrix(grad_out, "grad_out")[2]


_CURRENT = contextlib.nullcontext()


def _on(stream):
    """A context whose allocations belong to the stream that the work runs on."""
    return _CURRENT if stream is None else _torch.cuda.stream(stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


# ------------------------------------------------------------ distillation
def _distill(logits, top_values, top_indices, temperature, weights, losses, lse, grad, with_grad,
             backward, grad_losses, stream, wait_timeout_ns=0, status=None):
    torch = _torch or _load()
    kind, top_kind = _kind(logits, "logits"), _kind(top_values, "top_values")
    rows, cols, stride = _matrix(logits, "logits")
    top_rows, k, values_stride = _matrix(top_values, "top_values")
    if top_rows != rows or top_indices.shape != (rows, k):
        raise ValueError("top_values and top_indices must both have shape (rows, k)")
    indices_stride = _matrix(top_indices, "top_indices")[2]
    if not 1 <= k <= MAX_TOP:
        raise ValueError(f"1 to {MAX_TOP} top logits per row, got {k}")
    ib = _index_bytes(top_indices, "top_indices")
    if weights is not None:
        _vector(weights, rows, "weights")
    if losses is not None:
        _vector(losses, rows, "losses_out")
    if lse is not None:
        _vector(lse, rows, "lse" if backward else "lse_out")
    elif backward:
        raise ValueError("the backward call needs the forward call's lse")
    if grad_losses is not None:
        _vector(grad_losses, rows, "grad_losses")
    if status is not None:
        _vector(status, 1, "status_out", torch.int32)
    grad_stride = cols if grad is None else _grad_stride(logits, grad)
    index = _device(stream, logits, top_values, top_indices, weights, losses, lse, grad,
                    grad_losses, status)

    with _on(stream):
        device = logits.device
        if lse is None:
            lse = torch.empty((rows,), dtype=torch.float32, device=device)
        if losses is None and not backward:
            losses = torch.empty((rows,), dtype=torch.float32, device=device)
        if grad is None and with_grad:
            grad = torch.empty((rows, cols), dtype=logits.dtype, device=device)
    args = DistillArgs(logits.data_ptr(), stride, rows, cols, top_values.data_ptr(), values_stride,
                       top_indices.data_ptr(), indices_stride, _ptr(weights), _ptr(losses),
                       lse.data_ptr(), _ptr(grad), grad_stride, kind, top_kind, ib, k, temperature,
                       wait_timeout_ns, _ptr(status))
    lib = _lib_of()
    s = _raw_stream(index) if stream is None else stream.cuda_stream
    if backward:
        _check(lib.rs_distill_loss_backward(ctypes.byref(args), _ptr(grad_losses), s),
               "rs_distill_loss_backward")
        return grad
    _check(lib.rs_distill_loss(ctypes.byref(args), s), "rs_distill_loss")
    return (losses, lse, grad) if with_grad else (losses, lse)


def distill_loss(logits, top_values, top_indices, temperature: float = 1.0, weights=None,
                 losses_out=None, lse_out=None, stream=None):
    """(losses, lse) of a student's logits against its teacher's top logits.

    ``logits`` is (rows, cols) float16/bfloat16/float32; ``top_values`` and
    ``top_indices`` (int32/int64) are (rows, k), k <= 1024, with entries of an
    index outside [0, cols) not taking part.  ``losses`` are weights *
    temperature^2 * KL(teacher's softmax over its entries || student);
    ``lse`` is each row's log-sum-exp of logits / temperature, which
    ``distill_loss_backward`` takes.  Differentiable in ``logits``."""
    if _wants_grad(logits, stream, losses_out, lse_out):
        return _autograd().Distill.apply(logits, top_values, top_indices, float(temperature),
                                         weights)
    return _distill(logits, top_values, top_indices, temperature, weights, losses_out, lse_out,
                    None, False, False, None, stream)


def distill_loss_grad(logits, top_values, top_indices, temperature: float = 1.0, weights=None,
                      losses_out=None, lse_out=None, grad_out=None, stream=None,
                      wait_timeout_ns: int = 0, status_out=None):
    """(losses, lse, grad): ``distill_loss`` and the gradient of the sum of its
    losses.  ``grad_out`` may be ``logits`` itself.  ``wait_timeout_ns`` limits
    a wait inside the kernel of long rows (0: 2 s); where one runs out, rows
    that are not finished get NaN and ``status_out`` (one int32 on the device,
    zero beforehand) RS_ERR_LOOKBACK_TIMEOUT."""
    return _distill(logits, top_values, top_indices, temperature, weights, losses_out, lse_out,
                    grad_out, True, False, None, stream, wait_timeout_ns, status_out)


def distill_loss_backward(grad_losses, logits, lse, top_values, top_indices,
                          temperature: float = 1.0, weights=None, grad_out=None, stream=None):
    """Gradient of sum(grad_losses * losses) (None: ones) in ``logits``, with
    the ``lse`` of the forward call.  ``grad_out`` may be ``logits`` itself."""
    return _distill(logits, top_values, top_indices, temperature, weights, None, lse, grad_out,
                    True, True, grad_losses, stream)


# ------------------------------------------------------------- policy loss
def _policy(logits, actions, old, advantages, ref, clip_low, clip_high, kl_coef, temperature,
            weights, losses, logprobs, lse, grad, with_grad, backward, grad_losses, stream,
            wait_timeout_ns=0, status=None):
    torch = _torch or _load()
    kind = _kind(logits, "logits")
    rows, cols, stride = _matrix(logits, "logits")
    ib = _index_bytes(actions, "actions")
    _vector(actions, rows, "actions", actions.dtype)
    _vector(old, rows, "old_logprobs")
    _vector(advantages, rows, "advantages")
    if ref is not None:
        _vector(ref, rows, "ref_logprobs")
    elif kl_coef != 0:
        raise ValueError("a KL term needs ref_logprobs")
    if weights is not None:
        _vector(weights, rows, "weights")
    if losses is not None:
        _vector(losses, rows, "losses_out")
    if logprobs is not None:
        _vector(logprobs, rows, "logprobs_out")
    if lse is not None:
        _vector(lse, rows, "lse" if backward else "lse_out")
    elif backward:
        raise ValueError("the backward call needs the forward call's lse")
    if grad_losses is not None:
        _vector(grad_losses, rows, "grad_losses")
    if status is not None:
        _vector(status, 1, "status_out", torch.int32)
    grad_stride = cols if grad is None else _grad_stride(logits, grad)
    index = _device(stream, logits, actions, old, advantages, ref, weights, losses, logprobs, lse,
                    grad, grad_losses, status)

    with _on(stream):
        device = logits.device
        if lse is None:
            lse = torch.empty((rows,), dtype=torch.float32, device=device)
        if losses is None and not backward:
            losses = torch.empty((rows,), dtype=torch.float32, device=device)
        if logprobs is None and not backward:
            logprobs = torch.empty((rows,), dtype=torch.float32, device=device)
        if grad is None and with_grad:
            grad = torch.empty((rows, cols), dtype=logits.dtype, device=device)
    args = PolicyArgs(logits.data_ptr(), stride, rows, cols, actions.data_ptr(), old.data_ptr(),
                      advantages.data_ptr(), _ptr(ref), _ptr(weights), _ptr(losses),
                      _ptr(logprobs), lse.data_ptr(), _ptr(grad), grad_stride, kind, ib, clip_low,
                      clip_high, kl_coef, temperature, wait_timeout_ns, _ptr(status))
    lib = _lib_of()
    s = _raw_stream(index) if stream is None else stream.cuda_stream
    if backward:
        _check(lib.rs_policy_loss_backward(ctypes.byref(args), _ptr(grad_losses), s),
               "rs_policy_loss_backward")
        return grad
    _check(lib.rs_policy_loss(ctypes.byref(args), s), "rs_policy_loss")
    return (losses, logprobs, lse, grad) if with_grad else (losses, logprobs, lse)


def policy_loss(logits, actions, old_logprobs, advantages, ref_logprobs=None,
                clip_low: float = 0.2, clip_high: float = 0.2, kl_coef: float = 0.0,
                temperature: float = 1.0, weights=None, losses_out=None, logprobs_out=None,
                lse_out=None, stream=None):
    """(losses, logprobs, lse) of the clipped policy loss, one action per row.

    ``actions`` (int32/int64) holds the sampled column of each row (outside
    [0, cols): the row takes no part), ``old_logprobs`` its log-probability
    when it was sampled, ``ref_logprobs`` the reference policy's (needed when
    ``kl_coef`` is not 0).  ``logprobs`` are the present ones.  Differentiable
    in ``logits`` through ``losses``."""
    if _wants_grad(logits, stream, losses_out, logprobs_out, lse_out):
        return _autograd().Policy.apply(logits, actions, old_logprobs, advantages, ref_logprobs,
                                        float(clip_low), float(clip_high), float(kl_coef),
                                        float(temperature), weights)
    return _policy(logits, actions, old_logprobs, advantages, ref_logprobs, clip_low, clip_high,
                   kl_coef, temperature, weights, losses_out, logprobs_out, lse_out, None, False,
                   False, None, stream)


def policy_loss_grad(logits, actions, old_logprobs, advantages, ref_logprobs=None,
                     clip_low: float = 0.2, clip_high: float = 0.2, kl_coef: float = 0.0,
                     temperature: float = 1.0, weights=None, losses_out=None, logprobs_out=None,
                     lse_out=None, grad_out=None, stream=None, wait_timeout_ns: int = 0,
                     status_out=None):
    """(losses, logprobs, lse, grad): ``policy_loss`` and the gradient of the
    sum of its losses.  ``grad_out`` may be ``logits`` itself;
    ``wait_timeout_ns`` and ``status_out`` as ``distill_loss_grad``."""
    return _policy(logits, actions, old_logprobs, advantages, ref_logprobs, clip_low, clip_high,
                   kl_coef, temperature, weights, losses_out, logprobs_out, lse_out, grad_out,
                   True, False, None, stream, wait_timeout_ns, status_out)


def policy_loss_backward(grad_losses, logits, lse, actions, old_logprobs, advantages,
                         ref_logprobs=None, clip_low: float = 0.2, clip_high: float = 0.2,
                         kl_coef: float = 0.0, temperature: float = 1.0, weights=None,
                         grad_out=None, stream=None):
    """Gradient of sum(grad_losses * losses) (None: ones) in ``logits``, with
    the ``lse`` of the forward call.  ``grad_out`` may be ``logits`` itself."""
    return _policy(logits, actions, old_logprobs, advantages, ref_logprobs, clip_low, clip_high,
                   kl_coef, temperature, weights, None, None, lse, grad_out, True, True,
                   grad_losses, stream)


# ------------------------------------------------------------ balance loss
@functools.lru_cache(maxsize=256)
def balance_temp_bytes(tokens: int, experts: int) -> int:
    """Scratch size of ``balance_loss`` and ``balance_loss_grad``."""
    out = ctypes.c_size_t(0)
    _check(_lib_of().rs_balance_temp_bytes(tokens, experts, ctypes.byref(out)),
           "rs_balance_temp_bytes")
    return out.value


def _mask(mask, tokens):
    if mask.dtype not in (_torch.bool, _torch.uint8) or mask.shape != (tokens,):
        raise ValueError(f"token_mask must be bool or uint8 of shape ({tokens},)")
    if tokens > 1 and mask.stride(0) != 1:
        raise ValueError("token_mask must be contiguous")


def _balance(scores, ids, mask, scale, grad, with_grad, temp, stream):
    torch = _torch or _load()
    kind = _kind(scores, "scores")
    tokens, experts, stride = _matrix(scores, "scores")
    if ids.dim() != 2 or ids.shape[0] != tokens or ids.shape[1] < 1:
        raise ValueError("expert_ids must have shape (tokens, k), k >= 1")
    _, k, ids_stride = _matrix(ids, "expert_ids")
    ib = _index_bytes(ids, "expert_ids")
    if not 1 <= experts <= MAX_EXPERTS:
        raise ValueError(f"1 to {MAX_EXPERTS} experts, got {experts}")
    if mask is not None:
        _mask(mask, tokens)
    grad_stride = experts if grad is None else _grad_stride(scores, grad)
    index = _device(stream, scores, ids, mask, grad, temp)
    need = balance_temp_bytes(tokens, experts)
    with _on(stream):
        device = scores.device
        loss = torch.empty((), dtype=torch.float32, device=device)
        mean = torch.empty((experts,), dtype=torch.float32, device=device)
        counts = torch.empty((experts,), dtype=torch.int32, device=device)
        n = torch.empty((1,), dtype=torch.int32, device=device)
        if temp is None and need:
            temp = torch.empty((need,), dtype=torch.uint8, device=device)
        if grad is None and with_grad:
            grad = torch.empty((tokens, experts), dtype=scores.dtype, device=device)
    args = BalanceArgs(scores.data_ptr(), stride, tokens, ids.data_ptr(), ids_stride, _ptr(mask),
                       loss.data_ptr(), mean.data_ptr(), counts.data_ptr(), n.data_ptr(),
                       _ptr(grad), grad_stride, _ptr(temp),
                       0 if temp is None else temp.numel() * temp.element_size(),
                       kind, experts, ib, k, scale)
    s = _raw_stream(index) if stream is None else stream.cuda_stream
    _check(_lib_of().rs_balance_loss(ctypes.byref(args), s), "rs_balance_loss")
    return (loss, counts, mean, n, grad) if with_grad else (loss, counts, mean, n)


def balance_loss(scores, expert_ids, token_mask=None, temp=None, stream=None):
    """(loss, counts, mean_probs, n_tokens) of a router's load balance.

    ``scores`` is (tokens, experts <= 1024), ``expert_ids`` (int32/int64)
    (tokens, k): the experts chosen for each token, ids outside [0, experts)
    being dropped slots.  ``token_mask`` (bool) keeps the tokens that count.
    ``loss`` = experts * sum_e f_e P_e with f the experts' shares of the
    tokens * k slots and P their mean probabilities; ``counts`` are int32.
    Differentiable in ``scores`` through ``loss``."""
    if _wants_grad(scores, stream):
        return _autograd().Balance.apply(scores, expert_ids, token_mask, temp)
    return _balance(scores, expert_ids, token_mask, 1.0, None, False, temp, stream)


def balance_loss_grad(scores, expert_ids, token_mask=None, scale: float = 1.0, grad_out=None,
                      temp=None, stream=None):
    """(loss, counts, mean_probs, n_tokens, grad): ``balance_loss`` and the
    gradient of scale * loss.  ``grad_out`` may be ``scores`` itself."""
    return _balance(scores, expert_ids, token_mask, scale, grad_out, True, temp, stream)


def balance_loss_backward(grad_loss, scores, counts, n_tokens, top_k: int, token_mask=None,
                          grad_out=None, stream=None):
    """Gradient of grad_loss * loss in ``scores`` (``grad_loss``: one float32 on
    the device, None: 1), with the ``counts`` and ``n_tokens`` of the forward
    call, whose expert ids had ``top_k`` columns."""
    torch = _torch or _load()
    kind = _kind(scores, "scores")
    tokens, experts, stride = _matrix(scores, "scores")
    if not 1 <= experts <= MAX_EXPERTS:
        raise ValueError(f"1 to {MAX_EXPERTS} experts, got {experts}")
    if top_k < 1:
        raise ValueError("top_k must be at least 1")
    _vector(counts, experts, "counts", torch.int32)
    _vector(n_tokens, 1, "n_tokens", torch.int32)
    if grad_loss is not None and (grad_loss.dtype is not torch.float32 or grad_loss.numel() != 1):
        raise ValueError("grad_loss must be one float32")
    if token_mask is not None:
        _mask(token_mask, tokens)
    grad_stride = experts if grad_out is None else _grad_stride(scores, grad_out)
    index = _device(stream, scores, counts, n_tokens, grad_loss, token_mask, grad_out)
    grad = grad_out
    if grad is None:
        with _on(stream):
            grad = torch.empty((tokens, experts), dtype=scores.dtype, device=scores.device)
    args = BalanceArgs(scores.data_ptr(), stride, tokens, None, 0, _ptr(token_mask), None, None,
                       counts.data_ptr(), n_tokens.data_ptr(), grad.data_ptr(), grad_stride, None,
                       0, kind, experts, 0, top_k, 1.0)
    s = _raw_stream(index) if stream is None else stream.cuda_stream
    _check(_lib_of().rs_balance_loss_backward(ctypes.byref(args), _ptr(grad_loss), s),
           "rs_balance_loss_backward")
    return grad


def row_wait_timeout_probe(timeout_ns: int, stream=None) -> int:
    """Run the long-row kernels' bounded wait on a barrier on which nothing
    arrives (rs_row_wait_timeout_probe); return its status."""
    torch = _torch or _load()
    word = torch.empty(1, dtype=torch.int32, device="cuda")
    result = ctypes.c_int(-1)
    s = _raw_stream(word.get_device()) if stream is None else stream.cuda_stream
    _check(_lib_of().rs_row_wait_timeout_probe(word.data_ptr(), int(timeout_ns), s,
                                               ctypes.byref(result)),
           "rs_row_wait_timeout_probe")
    return result.value


# --------------------------------------------------------------- autograd
def _wants_grad(x, stream, *outs):
    """Whether the call is recorded by autograd, which allocates the outputs and
    runs the backward call on the stream that was current in the forward one."""
    if not x.requires_grad or not (_torch or _load()).is_grad_enabled():
        return False
    if stream is not None or any(o is not None for o in outs):
        raise ValueError("outputs or a stream cannot be given for scores that require a "
                         "gradient (use torch.cuda.stream)")
    return True


_FUNCTIONS = None


def _autograd():
    """The autograd functions (made at the first use: torch is not needed to
    import the package)."""
    global _FUNCTIONS
    if _FUNCTIONS is not None:
        return _FUNCTIONS
    import torch
    from torch.autograd.function import once_differentiable

    class Distill(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, values, indices, temperature, weights):
            losses, lse = _distill(logits, values, indices, temperature, weights, None, None, None,
                                   False, False, None, None)
            ctx.save_for_backward(logits, values, indices, weights, lse)
            ctx.temperature = temperature
            ctx.mark_non_differentiable(lse)
            return losses, lse

        @staticmethod
        @once_differentiable
        def backward(ctx, up, _):
            logits, values, indices, weights, lse = ctx.saved_tensors
            grad = distill_loss_backward(up.float().contiguous(), logits, lse, values, indices,
                                         ctx.temperature, weights)
            return grad, None, None, None, None

    class Policy(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, actions, old, advantages, ref, low, high, kl, temperature,
                    weights):
            losses, logprobs, lse = _policy(logits, actions, old, advantages, ref, low, high, kl,
                                            temperature, weights, None, None, None, None, False,
                                            False, None, None)
            ctx.save_for_backward(logits, actions, old, advantages, ref, weights, lse)
            ctx.rest = low, high, kl, temperature
            ctx.mark_non_differentiable(logprobs, lse)
            return losses, logprobs, lse

        @staticmethod
        @once_differentiable
        def backward(ctx, up, *_):
            logits, actions, old, advantages, ref, weights, lse = ctx.saved_tensors
            low, high, kl, temperature = ctx.rest
            grad = policy_loss_backward(up.float().contiguous(), logits, lse, actions, old,
                                        advantages, ref, low, high, kl, temperature, weights)
            return (grad,) + (None,) * 9

    class Balance(torch.autograd.Function):
        @staticmethod
        def forward(ctx, scores, ids, mask, temp):
            loss, counts, mean, n = _balance(scores, ids, mask, 1.0, None, False, temp, None)
            ctx.save_for_backward(scores, counts, n, mask)
            ctx.top_k = ids.shape[1]
            ctx.mark_non_differentiable(counts, mean, n)
            return loss, counts, mean, n

        @staticmethod
        @once_differentiable
        def backward(ctx, up, *_):
            scores, counts, n, mask = ctx.saved_tensors
            grad = balance_loss_backward(up.float(), scores, counts, n, ctx.top_k, mask)
            return grad, None, None, None

    _FUNCTIONS = types.SimpleNamespace(Distill=Distill, Policy=Policy, Balance=Balance)
    return _FUNCTIONS
