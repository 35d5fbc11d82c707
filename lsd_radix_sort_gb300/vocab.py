"""The two ends of a vocabulary: binding of ``rs_token_logprobs`` and ``rs_embedding``.

``token_logprobs`` scores rows of logits: the log probabilities of given
tokens, the entropy, and the top alternatives.  It makes what the losses take:
``policy_loss``'s old and reference log probabilities, and the lists that
``distill_loss`` is taught by, without a sort of whole rows.  Its backward call
gives the entropy bonus and the penalty on the log-sum-exp that go with them.

``embedding`` looks up rows of a table; ``embedding_grad`` and
``embedding_grad_rows`` are its gradient, as a whole table or as the rows that
some token names, summed over tokens that are sorted by id.

The formulas, and what happens to padded tokens, -inf and NaN, are stated in
include/lsdrs.h.  As in the rest of the package the work is enqueued on
``stream`` (the current stream by default) and nothing synchronises; results
are allocated by torch on that stream unless given.  All calls capture into a
CUDA graph; a captured training step is best made of the explicit backward
calls, since torch's engine ties a leaf to the stream of the first graph that
used it, and a capture must not wait for a graph that is still alive outside.
"""
from __future__ import annotations

import ctypes
import functools
import math
import types
import typing

from . import _check, _lib_of
from . import losses as _l
from .losses import (_F, _I, _I64, _P, _SZ, MAX_TOP, _device, _grad_stride, _index_bytes, _kind,
                     _matrix, _on, _ptr, _room, _vector, _wants_grad)

__all__ = ["TokenLogprobs", "token_logprobs", "token_logprobs_temp_bytes",
           "token_logprobs_backward", "embedding", "embedding_grad", "embedding_grad_rows",
           "embedding_grad_temp_bytes"]

EMBED_TABLE, EMBED_ADD, EMBED_ROWS = range(3)


class LogprobsArgs(ctypes.Structure):
    """struct rs_logprobs_args of include/lsdrs.h."""
    _fields_ = [("logits", _P), ("logits_stride", _I64), ("rows", _I64), ("cols", _I64),
                ("tokens", _P), ("tokens_stride", _I64), ("logprobs", _P), ("entropy", _P),
                ("lse", _P), ("stats", _P), ("top_logprobs", _P), ("top_ids", _P), ("grad", _P),
                ("grad_stride", _I64), ("temp", _P), ("temp_bytes", _SZ), ("logits_type", _I),
                ("index_bytes", _I), ("n_tokens", _I), ("top", _I), ("temperature", _F)]


class EmbeddingArgs(ctypes.Structure):
    """struct rs_embedding_args of include/lsdrs.h."""
    _fields_ = [("table", _P), ("table_stride", _I64), ("vocab", _I64), ("width", _I64),
                ("ids", _P), ("tokens", _I64), ("out", _P), ("out_stride", _I64), ("type", _I),
                ("index_bytes", _I), ("scale", _F)]


class EmbeddingGradArgs(ctypes.Structure):
    """struct rs_embedding_grad_args of include/lsdrs.h."""
    _fields_ = [("grad", _P), ("grad_stride", _I64), ("tokens", _I64), ("width", _I64),
                ("vocab", _I64), ("ids", _P), ("padding_id", _I64), ("out", _P),
                ("out_stride", _I64), ("row_ids", _P), ("count", _P), ("temp", _P),
                ("temp_bytes", _SZ), ("status", _P), ("grad_type", _I), ("out_type", _I),
                ("index_bytes", _I), ("mode", _I), ("scale", _F)]


class TokenLogprobs(typing.NamedTuple):
    """What ``token_logprobs`` returns; None for what was not asked for."""
    logprobs: typing.Any      # shape of tokens
    entropy: typing.Any       # (rows,)
    lse: typing.Any           # (rows,)
    top_logprobs: typing.Any  # (rows, top)
    top_ids: typing.Any       # (rows, top) int64
    stats: typing.Any         # (rows, 2): what the backward call takes


# -------------------------------------------------------- log probabilities
def _tokens_of(tokens, rows):
    """(columns, elements from one row to the next, bytes of one) of the tokens."""
    if tokens is None:
        return 0, 0, 8
    ib = _index_bytes(tokens, "tokens")
    if tokens.dim() == 1:
        _vector(tokens, rows, "tokens", tokens.dtype)
        return 1, 1, ib
    token_rows, k, stride = _matrix(tokens, "tokens")
    if token_rows != rows:
        raise ValueError(f"tokens must have shape ({rows},) or ({rows}, k)")
    if k > MAX_TOP:
        raise ValueError(f"at most {MAX_TOP} tokens per row, got {k}")
    return k, stride, ib


def _dense(t, shape, what, dtype=None):
    dtype = _l._torch.float32 if dtype is None else dtype
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous {dtype} of shape {tuple(shape)}, got "
                         f"{t.dtype} of {tuple(t.shape)}")


def token_logprobs_temp_bytes(rows: int, cols: int, logits_type: int, top: int = 0) -> int:
    """Scratch size of ``token_logprobs`` on the current device, for logits of
    an rs_score_type (0 float16, 1 bfloat16, 2 float32)."""
    n = ctypes.c_size_t(0)
    _check(_lib_of().rs_token_logprobs_temp_bytes(rows, cols, logits_type, top, ctypes.byref(n)),
           "rs_token_logprobs_temp_bytes")
    return n.value


@functools.lru_cache(maxsize=256)
def _logprobs_scratch(index, rows, cols, kind, top):
    """The same, kept for each device: the sizes go with its number of SMs."""
    return token_logprobs_temp_bytes(rows, cols, kind, top)


def _logprobs(logits, tokens, top, temperature, temp, stream):
    torch = _l._torch or _l._load()
    kind = _kind(logits, "logits")
    rows, cols, stride = _matrix(logits, "logits")
    k, token_stride, ib = _tokens_of(tokens, rows)
    if not 0 <= top <= MAX_TOP:
        raise ValueError(f"0 to {MAX_TOP} top alternatives per row, got {top}")
    index = _device(stream, logits, tokens, temp)
    need = _logprobs_scratch(index, rows, cols, kind, top)
    with _on(stream):
        device, f32 = logits.device, torch.float32
        logprobs = None if tokens is None else torch.empty(tokens.shape, dtype=f32, device=device)
        entropy = torch.empty((rows,), dtype=f32, device=device)
        lse = torch.empty((rows,), dtype=f32, device=device)
        stats = torch.empty((rows, 2), dtype=f32, device=device)
        top_logprobs = top_ids = None
        if top:
            top_logprobs = torch.empty((rows, top), dtype=f32, device=device)
            top_ids = torch.empty((rows, top), dtype=torch.int64, device=device)
        if temp is None:
            temp = torch.empty((need,), dtype=torch.uint8, device=device)
    args = LogprobsArgs(logits.data_ptr(), stride, rows, cols, _ptr(tokens), token_stride,
                        _ptr(logprobs), entropy.data_ptr(), lse.data_ptr(), stats.data_ptr(),
                        _ptr(top_logprobs), _ptr(top_ids), None, 0,
                        temp.data_ptr(), _room(temp), kind, ib, k, top,
                        temperature)
    s = _l._raw_stream(index) if stream is None else stream.cuda_stream
    _check(_lib_of().rs_token_logprobs(ctypes.byref(args), s), "rs_token_logprobs")
    return TokenLogprobs(logprobs, entropy, lse, top_logprobs, top_ids, stats)


def token_logprobs(logits, tokens=None, top: int = 0, temperature: float = 1.0, temp=None,
                   stream=None):
    """TokenLogprobs(logprobs, entropy, lse, top_logprobs, top_ids, stats) of rows of logits.

    ``logits`` is (rows, cols) float16/bfloat16/float32; ``tokens`` (int32/
    int64, (rows,) or (rows, k), k <= 1024) the columns whose log
    probabilities under softmax(logits / temperature) are wanted; one outside
    [0, cols) is a padded place and gets 0.  ``top`` (<= 1024) asks for that
    many alternatives: the columns of largest score, the best first, of equal
    ones the lower.  All but ``top_ids`` and ``stats`` are differentiable in
    ``logits``."""
    if _wants_grad(logits, stream, temp):
        return TokenLogprobs(*_autograd().Logprobs.apply(logits, tokens, int(top),
                                                         float(temperature)))
    return _logprobs(logits, tokens, top, temperature, temp, stream)


def token_logprobs_backward(logits, stats, entropy=None, tokens=None, top_ids=None,
                            grad_logprobs=None, grad_entropy=None, grad_lse=None, grad_top=None,
                            temperature: float = 1.0, grad_out=None, stream=None):
    """Gradient in ``logits`` of the sums of ``grad_logprobs`` * logprobs,
    ``grad_entropy`` * entropy, ``grad_lse`` * lse and ``grad_top`` *
    top_logprobs (each may be None), with ``stats``, ``entropy`` and
    ``top_ids`` of the forward call.  ``grad_out`` may be ``logits`` itself."""
    torch = _l._torch or _l._load()
    kind = _kind(logits, "logits")
    rows, cols, stride = _matrix(logits, "logits")
    k, token_stride, ib = _tokens_of(tokens, rows)
    _dense(stats, (rows, 2), "stats")
    top = 0
    if grad_logprobs is not None:
        if tokens is None:
            raise ValueError("grad_logprobs needs the tokens")
        _dense(grad_logprobs, tokens.shape, "grad_logprobs")
    if grad_entropy is not None:
        if entropy is None:
            raise ValueError("grad_entropy needs the forward call's entropy")
        _vector(entropy, rows, "entropy")
        _vector(grad_entropy, rows, "grad_entropy")
    if grad_lse is not None:
        _vector(grad_lse, rows, "grad_lse")
    if grad_top is not None:
        if top_ids is None or top_ids.dim() != 2:
            raise ValueError("grad_top needs the forward call's top_ids")
        top = top_ids.shape[1]
        if top > MAX_TOP:
            raise ValueError(f"0 to {MAX_TOP} top alternatives per row, got {top}")
        _dense(top_ids, (rows, top), "top_ids", torch.int64)
        _dense(grad_top, (rows, top), "grad_top")
    grad_stride = cols if grad_out is None else _grad_stride(logits, grad_out)
    index = _device(stream, logits, stats, entropy, tokens, top_ids, grad_logprobs, grad_entropy,
                    grad_lse, grad_top, grad_out)
    grad = grad_out
    if grad is None:
        with _on(stream):
            grad = torch.empty((rows, cols), dtype=logits.dtype, device=logits.device)
    args = LogprobsArgs(logits.data_ptr(), stride, rows, cols, _ptr(tokens), token_stride, None,
                        _ptr(entropy), None, stats.data_ptr(), None,
                        _ptr(top_ids) if top else None, grad.data_ptr(), grad_stride, None, 0,
                        kind, ib, k, top, temperature)
    s = _l._raw_stream(index) if stream is None else stream.cuda_stream
    _check(_lib_of().rs_token_logprobs_backward(
        ctypes.byref(args), _ptr(grad_logprobs) if k else None, _ptr(grad_entropy),
        _ptr(grad_lse), _ptr(grad_top) if top else None, s), "rs_token_logprobs_backward")
    return grad


# ----------------------------------------------------------------- embedding
def _ids_of(ids):
    ib = _index_bytes(ids, "ids")
    if not ids.is_contiguous():
        raise ValueError("ids must be contiguous")
    return ids.numel(), ib


def _rows_of(t, ids, width, what):
    """Elements from one row to the next of a tensor of shape ids.shape + (width,)."""
    if t.shape != ids.shape + (width,):
        raise ValueError(f"{what} must have shape {tuple(ids.shape) + (width,)}, got "
                         f"{tuple(t.shape)}")
    if t.dim() == 2:
        return _matrix(t, what)[2]
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return width


def _scale(scale):
    if not math.isfinite(scale):
        raise ValueError(f"scale must be finite, got {scale}")
    return scale


def _padding_id(padding_id):
    if padding_id < -1:
        raise ValueError(f"padding_id must be an id, or -1 for none, got {padding_id}")
    return padding_id


def _embed(table, ids, scale, out, stream):
    torch = _l._torch or _l._load()
    kind = _kind(table, "table")
    vocab, width, table_stride = _matrix(table, "table")
    n, ib = _ids_of(ids)
    if vocab < 1 or width < 1:
        raise ValueError("table must have at least one row and one column")
    if out is not None and out.dtype is not table.dtype:
        raise TypeError(f"out must be {table.dtype}, got {out.dtype}")
    out_stride = width if out is None else _rows_of(out, ids, width, "out")
    index = _device(stream, table, ids, out)
    if out is None:
        with _on(stream):
            out = torch.empty(ids.shape + (width,), dtype=table.dtype, device=table.device)
    args = EmbeddingArgs(table.data_ptr(), table_stride, vocab, width, ids.data_ptr(), n,
                         out.data_ptr(), out_stride, kind, ib, _scale(scale))
    s = _l._raw_stream(index) if stream is None else stream.cuda_stream
    _check(_lib_of().rs_embedding(ctypes.byref(args), s), "rs_embedding")
    return out


def embedding(table, ids, scale: float = 1.0, padding_id: int = -1, out=None, stream=None):
    """``scale`` * ``table[ids]``, of shape ids.shape + (width,) and the table's type.

    ``table`` is (vocab, width) float16/bfloat16/float32, ``ids`` int32/int64
    of any shape; an id outside [0, vocab) gives zeros.  Differentiable in
    ``table``; tokens of ``padding_id`` are looked up like any other, but take
    no part in the gradient."""
    _padding_id(padding_id)
    if _wants_grad(table, stream, out):
        return _autograd().Embedding.apply(table, ids, float(scale), int(padding_id))
    return _embed(table, ids, scale, out, stream)


@functools.lru_cache(maxsize=256)
def embedding_grad_temp_bytes(tokens: int, vocab: int, width: int) -> int:
    """Scratch size of ``embedding_grad`` and ``embedding_grad_rows``."""
    n = ctypes.c_size_t(0)
    _check(_lib_of().rs_embedding_grad_temp_bytes(tokens, vocab, width, ctypes.byref(n)),
           "rs_embedding_grad_temp_bytes")
    return n.value


def _embed_grad(grad, ids, vocab, scale, padding_id, dtype, out, mode, row_ids, count, temp,
                status, stream):
    torch = _l._torch or _l._load()
    kind = _kind(grad, "grad")
    n, ib = _ids_of(ids)
    if grad.dim() < 1 or grad.shape[-1] < 1:
        raise ValueError("grad must have shape ids.shape + (width,)")
    width = grad.shape[-1]
    grad_stride = _rows_of(grad, ids, width, "grad")
    if not 1 <= vocab < 1 << 31:
        raise ValueError(f"vocab must be from 1 to 2^31 - 1, got {vocab}")
    _padding_id(padding_id)
    if dtype is None:
        dtype = grad.dtype if out is None else out.dtype
    if dtype is not grad.dtype and dtype is not torch.float32:
        raise TypeError(f"the gradient of {grad.dtype} is {grad.dtype} or float32, not {dtype}")
    rows = min(n, vocab) if mode == EMBED_ROWS else vocab
    out_stride = width
    if out is not None:
        if out.dtype is not dtype or out.shape != (rows, width):
            raise ValueError(f"the output must be {dtype} of shape ({rows}, {width}), got "
                             f"{out.dtype} of {tuple(out.shape)}")
        out_stride = _matrix(out, "the output")[2]
    if row_ids is not None:
        _vector(row_ids, rows, "row_ids_out", torch.int64)
    if count is not None:
        _vector(count, 1, "count_out", torch.int32)
    if status is not None:
        _vector(status, 1, "status_out", torch.int32)
    index = _device(stream, grad, ids, out, row_ids, count, temp, status)
    need = embedding_grad_temp_bytes(n, vocab, width)
    with _on(stream):
        device = grad.device
        if out is None:
            out = torch.empty((rows, width), dtype=dtype, device=device)
        if mode == EMBED_ROWS:
            if row_ids is None:
                row_ids = torch.empty((rows,), dtype=torch.int64, device=device)
            if count is None:
                count = torch.empty((1,), dtype=torch.int32, device=device)
        if temp is None:
            temp = torch.empty((need,), dtype=torch.uint8, device=device)
    args = EmbeddingGradArgs(grad.data_ptr(), grad_stride, n, width, vocab, ids.data_ptr(),
                             padding_id, out.data_ptr(), out_stride, _ptr(row_ids), _ptr(count),
                             temp.data_ptr(), _room(temp), _ptr(status),
                             kind, _l._TYPES[dtype], ib, mode, _scale(scale))
    s = _l._raw_stream(index) if stream is None else stream.cuda_stream
    _check(_lib_of().rs_embedding_grad(ctypes.byref(args), s), "rs_embedding_grad")
    return (row_ids, out, count) if mode == EMBED_ROWS else out


def embedding_grad(grad, ids, vocab: int, scale: float = 1.0, padding_id: int = -1, dtype=None,
                   grad_out=None, accumulate: bool = False, temp=None, status_out=None,
                   stream=None):
    """The gradient of ``embedding`` in its table, (vocab, width).

    ``grad`` is the upstream gradient, of shape ids.shape + (width,); tokens of
    an id outside [0, vocab), or of ``padding_id``, take no part.  The result
    has ``dtype``: grad's type or float32.  With ``accumulate`` it is added to
    ``grad_out``, of which only rows that some token names are touched."""
    if accumulate and grad_out is None:
        raise ValueError("accumulate needs grad_out")
    return _embed_grad(grad, ids, vocab, scale, padding_id, dtype, grad_out,
                       EMBED_ADD if accumulate else EMBED_TABLE, None, None, temp, status_out,
                       stream)


def embedding_grad_rows(grad, ids, vocab: int, scale: float = 1.0, padding_id: int = -1,
                        dtype=None, row_ids_out=None, rows_out=None, count_out=None, temp=None,
                        status_out=None, stream=None):
    """(row_ids, rows, count): the rows of ``embedding_grad`` that some token
    names, in ascending order of their ids, for an optimizer that updates no
    others.  There is room for min(tokens, vocab) of them; ``count`` (int32, on
    the device) says how many there are, ``row_ids`` past it are -1 and
    ``rows`` past it are not written."""
    return _embed_grad(grad, ids, vocab, scale, padding_id, dtype, rows_out, EMBED_ROWS,
                       row_ids_out, count_out, temp, status_out, stream)


# ------------------------------------------------------------------ autograd
_FUNCTIONS = None


def _autograd():
    """The autograd functions (made at the first use: torch is not needed to
    import the package)."""
    global _FUNCTIONS
    if _FUNCTIONS is not None:
        return _FUNCTIONS
    import torch
    from torch.autograd.function import once_differentiable

    def flat(up):
        return None if up is None else up.float().contiguous()

    class Logprobs(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, tokens, top, temperature):
            got = _logprobs(logits, tokens, top, temperature, None, None)
            ctx.save_for_backward(logits, got.stats, got.entropy, tokens, got.top_ids)
            ctx.temperature = temperature
            ctx.set_materialize_grads(False)
            ctx.mark_non_differentiable(*(t for t in (got.top_ids, got.stats) if t is not None))
            return tuple(got)

        @staticmethod
        @once_differentiable
        def backward(ctx, up_logprobs, up_entropy, up_lse, up_top, *_):
            logits, stats, entropy, tokens, top_ids = ctx.saved_tensors
            ups = [flat(u) for u in (up_logprobs, up_entropy, up_lse, up_top)]
            if all(u is None for u in ups):
                return None, None, None, None
            grad = token_logprobs_backward(logits, stats, entropy, tokens, top_ids, *ups,
                                           temperature=ctx.temperature)
            return grad, None, None, None

    class Embedding(torch.autograd.Function):
        @staticmethod
        def forward(ctx, table, ids, scale, padding_id):
            ctx.save_for_backward(ids)
            ctx.rest = table.shape[0], scale, padding_id
            return _embed(table, ids, scale, None, None)

        @staticmethod
        @once_differentiable
        def backward(ctx, up):
            ids, = ctx.saved_tensors
            vocab, scale, padding_id = ctx.rest
            return embedding_grad(up.contiguous(), ids, vocab, scale, padding_id), None, None, None

    _FUNCTIONS = types.SimpleNamespace(Logprobs=Logprobs, Embedding=Embedding)
    return _FUNCTIONS
