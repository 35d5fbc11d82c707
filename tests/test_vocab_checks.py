"""What the log probabilities and the embedding refuse, before anything is
enqueued: by the binding (types, shapes, strides, devices) and by the C ABI."""
import ctypes

import pytest
import torch

import lsd_radix_sort_gb300 as rs
from lsd_radix_sort_gb300 import vocab


@pytest.fixture(scope="module")
def lib():
    from lsd_radix_sort_gb300 import build
    build.build()
    return rs.load_library()


def f(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


def i(*shape, dtype=torch.int64):
    return torch.zeros(*shape, dtype=dtype)


B = torch.bfloat16


@pytest.mark.parametrize("error,match,call", [
    (TypeError, "float16, bfloat16 or float32", lambda: rs.token_logprobs(f(4, 9, dtype=torch.float64))),
    (ValueError, "2-D", lambda: rs.token_logprobs(f(9))),
    (ValueError, "unit stride", lambda: rs.token_logprobs(f(9, 4).t())),
    (ValueError, "do not overlap", lambda: rs.token_logprobs(f(1, 9).expand(4, 9))),
    (TypeError, "int32 or int64", lambda: rs.token_logprobs(f(4, 9), i(4, dtype=torch.int16))),
    (ValueError, "tokens", lambda: rs.token_logprobs(f(4, 9), i(3))),
    (ValueError, "tokens must be contiguous", lambda: rs.token_logprobs(f(4, 9), i(8)[::2])),
    (ValueError, "tokens must have shape", lambda: rs.token_logprobs(f(4, 9), i(3, 2))),
    (ValueError, "2-D", lambda: rs.token_logprobs(f(4, 9), i(4, 1, 1))),
    (ValueError, "1024 tokens", lambda: rs.token_logprobs(f(4, 9), i(4, 1025))),
    (ValueError, "1024 top", lambda: rs.token_logprobs(f(4, 9), None, 1025)),
    (ValueError, "1024 top", lambda: rs.token_logprobs(f(4, 9), None, -1)),
    (ValueError, "CUDA device", lambda: rs.token_logprobs(f(4, 9), i(4), 2)),
    (ValueError, "cannot be given", lambda: rs.token_logprobs(f(4, 9).requires_grad_(True), stream=object())),
    (ValueError, "stats", lambda: rs.token_logprobs_backward(f(4, 9), f(4))),
    (ValueError, "stats", lambda: rs.token_logprobs_backward(f(4, 9), f(4, 2, dtype=B))),
    (ValueError, "needs the tokens", lambda: rs.token_logprobs_backward(f(4, 9), f(4, 2), grad_logprobs=f(4, 1))),
    (ValueError, "grad_logprobs must be", lambda: rs.token_logprobs_backward(f(4, 9), f(4, 2), tokens=i(4, 2), grad_logprobs=f(4, 1))),
    (ValueError, "grad_logprobs must be", lambda: rs.token_logprobs_backward(f(4, 9), f(4, 2), tokens=i(4, 2), grad_logprobs=f(2, 4).t())),
    (ValueError, "forward call's entropy", lambda: rs.token_logprobs_backward(f(4, 9), f(4, 2), grad_entropy=f(4))),
    (ValueError, "grad_entropy", lambda: rs.token_logprobs_backward(f(4, 9), f(4, 2), f(4), grad_entropy=f(3))),
    (ValueError, "grad_lse", lambda: rs.token_logprobs_backward(f(4, 9), f(4, 2), grad_lse=f(4, 1))),
    (ValueError, "forward call's top_ids", lambda: rs.token_logprobs_backward(f(4, 9), f(4, 2), grad_top=f(4, 2))),
    (ValueError, "top_ids must be", lambda: rs.token_logprobs_backward(f(4, 9), f(4, 2), top_ids=i(4, 2, dtype=torch.int32), grad_top=f(4, 2))),
    (ValueError, "grad_top must be", lambda: rs.token_logprobs_backward(f(4, 9), f(4, 2), top_ids=i(4, 2), grad_top=f(4, 3))),
    (ValueError, "1024 top", lambda: rs.token_logprobs_backward(f(4, 9), f(4, 2), top_ids=i(4, 1025), grad_top=f(4, 1025))),
    (ValueError, "grad_out must be", lambda: rs.token_logprobs_backward(f(4, 9), f(4, 2), grad_out=f(4, 9, dtype=B))),
    (ValueError, "CUDA device", lambda: rs.token_logprobs_backward(f(4, 9), f(4, 2))),
    (TypeError, "table must be", lambda: rs.embedding(i(4, 9), i(3))),
    (ValueError, "2-D", lambda: rs.embedding(f(9), i(3))),
    (ValueError, "unit stride", lambda: rs.embedding(f(9, 4).t(), i(3))),
    (ValueError, "at least one row", lambda: rs.embedding(f(0, 4), i(3))),
    (TypeError, "ids must be int32", lambda: rs.embedding(f(4, 9), f(3))),
    (ValueError, "ids must be contiguous", lambda: rs.embedding(f(4, 9), i(6)[::2])),
    (ValueError, "out must have shape", lambda: rs.embedding(f(4, 9), i(3), out=f(4, 9))),
    (ValueError, "out must have shape", lambda: rs.embedding(f(4, 9), i(2, 3), out=f(6, 9))),
    (ValueError, "out must be contiguous", lambda: rs.embedding(f(4, 9), i(2, 3), out=f(2, 3, 10)[..., :9])),
    (TypeError, "out must be", lambda: rs.embedding(f(4, 9), i(3), out=f(3, 9, dtype=B))),
    (ValueError, "CUDA device", lambda: rs.embedding(f(4, 9), i(3))),
    (ValueError, "cannot be given", lambda: rs.embedding(f(4, 9).requires_grad_(True), i(3), out=f(3, 9))),
    (TypeError, "grad must be", lambda: rs.embedding_grad(i(3, 9), i(3), 4)),
    (ValueError, "grad must have shape", lambda: rs.embedding_grad(f(4, 9), i(3), 4)),
    (ValueError, "grad must have shape", lambda: rs.embedding_grad(f(3, 0), i(3), 4)),
    (ValueError, "grad must be contiguous", lambda: rs.embedding_grad(f(3, 2, 10)[..., :9], i(3, 2), 4)),
    (ValueError, "vocab", lambda: rs.embedding_grad(f(3, 9), i(3), 0)),
    (ValueError, "vocab", lambda: rs.embedding_grad(f(3, 9), i(3), 1 << 31)),
    (ValueError, "padding_id", lambda: rs.embedding_grad(f(3, 9), i(3), 4, padding_id=-2)),
    (TypeError, "or float32", lambda: rs.embedding_grad(f(3, 9), i(3), 4, dtype=B)),
    (ValueError, "the output", lambda: rs.embedding_grad(f(3, 9), i(3), 4, grad_out=f(3, 9))),
    (ValueError, "the output", lambda: rs.embedding_grad(f(3, 9), i(3), 4, dtype=torch.float32, grad_out=f(4, 9, dtype=B))),
    (ValueError, "accumulate needs", lambda: rs.embedding_grad(f(3, 9), i(3), 4, accumulate=True)),
    (ValueError, "row_ids_out", lambda: rs.embedding_grad_rows(f(3, 9), i(3), 4, row_ids_out=i(4))),
    (ValueError, "the output", lambda: rs.embedding_grad_rows(f(3, 9), i(3), 4, rows_out=f(4, 9))),
    (ValueError, "the output", lambda: rs.embedding_grad_rows(f(5, 9), i(5), 4, rows_out=f(5, 9))),
    (ValueError, "count_out", lambda: rs.embedding_grad_rows(f(3, 9), i(3), 4, count_out=i(1))),
    (ValueError, "status_out", lambda: rs.embedding_grad(f(3, 9), i(3), 4, status_out=i(1))),
    (ValueError, "CUDA device", lambda: rs.embedding_grad(f(3, 9), i(3), 4)),
])
def test_binding_refuses(error, match, call):
    with pytest.raises(error, match=match):
        call()


CALLS = {
    "token_logprobs": lambda **kw: rs.token_logprobs(f(4, 9), i(4), 2, **kw),
    "token_logprobs_backward": lambda **kw: rs.token_logprobs_backward(f(4, 9), f(4, 2), **kw),
    "embedding": lambda **kw: rs.embedding(f(4, 9), i(3), **kw),
    "embedding_grad": lambda **kw: rs.embedding_grad(f(3, 9), i(3), 4, **kw),
    "embedding_grad_rows": lambda **kw: rs.embedding_grad_rows(f(3, 9), i(3), 4, **kw),
}


class OtherStream:
    device_index = 0
    cuda_stream = 0


@pytest.mark.parametrize("name", sorted(CALLS))
def test_tensors_of_a_device_that_is_not_current(monkeypatch, name):
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 1)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="current CUDA device, got cuda:1 while cuda:0"):
        CALLS[name]()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="the stream must be one of cuda:1"):
        CALLS[name](stream=OtherStream())


@pytest.mark.parametrize("scale", [float("nan"), float("inf")])
def test_scales_that_are_none(scale):
    with pytest.raises(ValueError, match="scale must be finite"):
        vocab._scale(scale)


def test_scratch_sizes_are_kept_for_each_device(monkeypatch):
    """Devices of unlike numbers of SMs divide the same rows differently."""
    on, asked = [0], []

    class Lib:
        @staticmethod
        def rs_token_logprobs_temp_bytes(rows, cols, kind, top, out):
            out._obj.value = 256 * (1 + on[0])
            return 0

        @staticmethod
        def rs_token_logprobs(args, stream):
            asked.append(args._obj.temp_bytes)
            return 0

    vocab._l._load()
    monkeypatch.setattr(vocab, "_lib_of", lambda: Lib)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: on[0])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: on[0])
    monkeypatch.setattr(vocab._l, "_raw_stream", lambda index: 0)
    for on[0] in (0, 1, 0, 1):
        rs.token_logprobs(f(4, 977))
        assert rs.token_logprobs_temp_bytes(4, 977, 2) == 256 * (1 + on[0])
    assert asked == [256, 512, 256, 512]


@pytest.mark.parametrize("call", [
    lambda **kw: rs.token_logprobs(f(4, 9), **kw), lambda **kw: rs.embedding_grad(f(3, 9), i(3), 4, **kw),
    lambda **kw: rs.embedding_grad_rows(f(3, 9), i(3), 4, **kw), lambda **kw: rs.balance_loss(f(4, 9), i(4, 2), **kw)])
def test_scratch_that_repeats_its_memory(lib, monkeypatch, call):
    """A megabyte by its shape, and one byte by its memory."""
    def reached(*args):
        raise AssertionError("the call was made")

    vocab._l._load()
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(vocab._l, "_raw_stream", reached)
    for temp in (i(1, dtype=torch.uint8).expand(1 << 20), i(1 << 20, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="temp must be contiguous"):
            call(temp=temp)


def test_forward_mode_is_refused():
    """A tangent is not dropped without a word, by the losses neither."""
    fwd = torch.autograd.forward_ad
    calls = [lambda x: rs.token_logprobs(x, i(4)), lambda x: rs.embedding(x, i(3)),
             lambda x: rs.distill_loss(x, f(4, 2), i(4, 2)), lambda x: rs.policy_loss(x, i(4), f(4), f(4)),
             lambda x: rs.balance_loss(x, i(4, 2))]
    for call in calls:
        for x in (f(4, 9), f(4, 9).requires_grad_(True)):
            with fwd.dual_level():
                dual = fwd.make_dual(x, f(4, 9))
                with pytest.raises(ValueError, match="no forward-mode derivatives"):
                    call(dual)
                with pytest.raises(ValueError, match="CUDA device"):
                    call(fwd.unpack_dual(dual).primal.detach())
            with pytest.raises(ValueError, match="no forward-mode derivatives"):
                torch.func.jvp(call, (x,), (f(4, 9),))


def test_a_padding_id_that_is_none_is_refused_before_the_backward_call():
    for table in (f(4, 9), f(4, 9).requires_grad_(True)):
        with pytest.raises(ValueError, match="padding_id must be an id"):
            rs.embedding(table, i(3), padding_id=-2)


# ------------------------------------------------------------------- the C ABI
BASE = 0x10000000  # addresses that no call here may touch
NAN, INF = float("nan"), float("inf")


def logprobs_args(**change):
    a = dict(logits=BASE, logits_stride=100, rows=4, cols=100, tokens=BASE + 0x100000,
             tokens_stride=2, logprobs=BASE + 0x200000, entropy=BASE + 0x210000,
             lse=BASE + 0x220000, stats=BASE + 0x230000, top_logprobs=BASE + 0x240000,
             top_ids=BASE + 0x250000, grad=BASE + 0x400000, grad_stride=100, temp=BASE + 0x500000,
             temp_bytes=1 << 30, logits_type=1,
             index_bytes=8, n_tokens=2, top=3, temperature=1.0)
    return vocab.LogprobsArgs(**{**a, **change})


SHARED = [dict(logits_type=3), dict(logits_type=-1), dict(rows=-1), dict(rows=1 << 31),
          dict(cols=0), dict(cols=1 << 30), dict(logits_stride=99), dict(logits_stride=1 << 61),
          dict(temperature=0.0), dict(temperature=-1.0), dict(temperature=NAN),
          dict(temperature=INF), dict(temperature=1e-45), dict(logits=None), dict(logits=BASE + 1),
          dict(index_bytes=2), dict(tokens=None), dict(tokens=BASE + 0x100004),
          dict(tokens_stride=1), dict(n_tokens=-1), dict(n_tokens=1025, tokens_stride=1025),
          dict(top=-1), dict(top=1025), dict(stats=None), dict(stats=BASE + 0x230004)]


@pytest.mark.parametrize("change", SHARED + [
    dict(logprobs=None), dict(logprobs=BASE + 2), dict(entropy=None), dict(lse=None),
    dict(top_logprobs=None), dict(top_ids=None), dict(top_ids=BASE + 0x250004), dict(temp=None),
    dict(temp=BASE + 0x500010)])
def test_logprobs_refuses(lib, change):
    assert lib.rs_token_logprobs(ctypes.byref(logprobs_args(**change)), None) == rs.RS_ERR_INVALID


@pytest.mark.parametrize("change", SHARED + [
    dict(grad=None), dict(grad=BASE + 0x400001), dict(grad=BASE + 2), dict(grad_stride=99),
    dict(grad=BASE, grad_stride=101), dict(entropy=None), dict(top_ids=None),
    dict(n_tokens=0), dict(top=0)])
def test_logprobs_backward_refuses(lib, change):
    up = [ctypes.c_void_p(BASE + 0x300000 + 0x10000 * n) for n in range(4)]
    call = lib.rs_token_logprobs_backward
    assert call(ctypes.byref(logprobs_args(**change)), *up, None) == rs.RS_ERR_INVALID
    for n in range(4):
        bad = up[:n] + [ctypes.c_void_p(BASE + 2)] + up[n + 1:]
        assert call(ctypes.byref(logprobs_args()), *bad, None) == rs.RS_ERR_INVALID


def embedding_args(**change):
    a = dict(table=BASE, table_stride=64, vocab=100, width=64, ids=BASE + 0x100000, tokens=8,
             out=BASE + 0x200000, out_stride=64, type=1, index_bytes=8, scale=1.0)
    return vocab.EmbeddingArgs(**{**a, **change})


@pytest.mark.parametrize("change", [
    dict(type=3), dict(type=-1), dict(index_bytes=2), dict(vocab=0), dict(vocab=1 << 31),
    dict(width=0), dict(tokens=-1), dict(tokens=1 << 31), dict(table_stride=63), dict(out_stride=63),
    dict(table=None), dict(table=BASE + 1), dict(ids=None), dict(ids=BASE + 0x100004),
    dict(out=None), dict(out=BASE + 0x200001), dict(out=BASE), dict(out=BASE + 64 * 99 * 2),
    dict(scale=NAN), dict(scale=INF)])
def test_embedding_refuses(lib, change):
    assert lib.rs_embedding(ctypes.byref(embedding_args(**change)), None) == rs.RS_ERR_INVALID


def grad_args(**change):
    a = dict(grad=BASE, grad_stride=64, tokens=8, width=64, vocab=100, ids=BASE + 0x100000,
             padding_id=-1, out=BASE + 0x200000, out_stride=64, row_ids=BASE + 0x300000,
             count=BASE + 0x310000, temp=BASE + 0x400000, temp_bytes=1 << 30, status=None,
             grad_type=1, out_type=1, index_bytes=8, mode=0, scale=1.0)
    return vocab.EmbeddingGradArgs(**{**a, **change})


@pytest.mark.parametrize("change,status", [
    (dict(grad_type=3), 1), (dict(out_type=0), 1), (dict(grad_type=2, out_type=1), 1),
    (dict(mode=3), 1), (dict(mode=-1), 1), (dict(index_bytes=1), 1), (dict(tokens=-1), 1),
    (dict(tokens=1 << 31), 1), (dict(vocab=0), 1), (dict(vocab=1 << 31), 1), (dict(width=0), 1),
    (dict(padding_id=-2), 1), (dict(scale=NAN), 1), (dict(grad_stride=63), 1),
    (dict(out_stride=63), 1), (dict(grad=None), 1), (dict(grad=BASE + 1), 1), (dict(ids=None), 1),
    (dict(ids=BASE + 0x100004), 1), (dict(out=None), 1), (dict(out=BASE + 0x200001), 1),
    (dict(out=BASE + 128), 1), (dict(out_type=2, out=BASE + 0x200002), 1),
    (dict(mode=2, row_ids=None), 1), (dict(mode=2, row_ids=BASE + 0x300004), 1),
    (dict(mode=2, count=None), 1), (dict(temp=None), 1), (dict(temp=BASE + 0x400010), 1),
    (dict(status=BASE + 2), 1), (dict(temp_bytes=255), 2)])
def test_embedding_grad_refuses(lib, change, status):
    assert lib.rs_embedding_grad(ctypes.byref(grad_args(**change)), None) == status


def test_no_work_and_no_arguments(lib):
    assert lib.rs_token_logprobs(ctypes.byref(logprobs_args(rows=0, logits=None, stats=None)), None) == 0
    assert lib.rs_token_logprobs_backward(ctypes.byref(logprobs_args(rows=0, grad=None)), None, None, None, None,
                                          None) == 0
    assert lib.rs_embedding(ctypes.byref(embedding_args(tokens=0, ids=None, out=None)), None) == 0
    assert lib.rs_token_logprobs(None, None) == 1 and lib.rs_embedding(None, None) == 1
    assert lib.rs_token_logprobs_backward(None, None, None, None, None, None) == 1
    assert lib.rs_embedding_grad(None, None) == 1


def test_scratch_size(lib):
    out = ctypes.c_size_t(0)
    for bad in ((-1, 8, 1, 0), (1 << 31, 8, 1, 0), (10, 0, 1, 0), (10, 1 << 30, 1, 0), (10, 8, 3, 0),
                (10, 8, 1, -1), (10, 8, 1, 1025)):
        assert lib.rs_token_logprobs_temp_bytes(*bad, ctypes.byref(out)) == 1
    assert lib.rs_token_logprobs_temp_bytes(10, 8, 1, 0, None) == 1
    for bad in ((-1, 8, 8), (1 << 31, 8, 8), (10, 0, 8), (10, 1 << 31, 8), (10, 8, 0), (10, 8, (1 << 24) + 1)):
        assert lib.rs_embedding_grad_temp_bytes(*bad, ctypes.byref(out)) == 1
    assert lib.rs_embedding_grad_temp_bytes(10, 8, 8, None) == 1
    assert rs.embedding_grad_temp_bytes(100000, 1000, 64) > rs.embedding_grad_temp_bytes(1000, 1000, 64) > 0


def test_scratch_of_a_gradient_is_a_fraction_of_it(lib):
    """Two sums of 32-bit columns for 32 tokens, a few counters, and the list of
    16 bytes a token (beyond 65,536 tokens the sort's as well)."""
    for tokens, width in ((32768, 4096), (65536, 8), (65536, 2047), (100000, 1024)):
        columns = -(-width // (512 if width % 16 == 0 else 256)) * (512 if width % 16 == 0 else 256)
        places = 2 * -(-tokens // 32)
        rest = 24 * tokens if tokens <= 65536 else 60 * tokens + (1 << 22)
        assert rs.embedding_grad_temp_bytes(tokens, 131072, width) <= places * (columns + columns // 64) * 4 + rest
