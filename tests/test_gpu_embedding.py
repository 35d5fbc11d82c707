"""Embedding lookup and its gradient against their formulas in 64 bits: types,
widths and alignments, ids that are missing, outside, padded or all alike,
whole tables, sums, rows; streams, graphs, and the same bits in every run."""
import math

import pytest
import torch

from tests import vocab_oracle as vo
from tests.loss_bounds import within

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]
WIDTHS = [1, 2, 3, 7, 8, 31, 64, 100, 257, 1000, 2056]


def randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def ids_of(g, n, vocab, kind="some"):
    """Tokens as text has them: few ids make up most; or each different."""
    if kind == "all":
        return torch.randint(0, vocab, (n,), generator=g, device="cuda")
    r = torch.rand(n, generator=g, device="cuda")
    return (vocab ** r - 1).long().clamp(0, vocab - 1)


def lookup(table, ids, scale):
    live = (ids >= 0) & (ids < table.shape[0])
    rows = (table[torch.where(live, ids, 0).long()].float() * scale).to(table.dtype)
    return torch.where(live[..., None], rows, torch.zeros_like(rows))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", WIDTHS)
def test_lookup(rs, width, dtype):
    g = gen(width)
    table = randn(g, 301, width, dtype=dtype)
    for n in (0, 1, 5, 700):
        ids = ids_of(g, n, 301)
        ids[1:n:5] = -1
        ids[2:n:7] = 301
        for scale in (1.0, math.sqrt(width), 0.0, -2.5):
            for index in (ids, ids.int()):
                assert torch.equal(rs.embedding(table, index, scale), lookup(table, ids, scale))
    far = torch.tensor([2 ** 40, -2 ** 40, 3], device="cuda")
    assert torch.equal(rs.embedding(table, far), lookup(table, far, 1.0))


@pytest.mark.parametrize("dtype", TYPES)
def test_lookup_shapes_strides_and_alignments(rs, dtype):
    g = gen(1)
    ids = ids_of(g, 60, 50).reshape(3, 4, 5)
    for width, pad, shift in ((64, 0, 0), (64, 8, 8), (64, 2, 2), (64, 1, 1), (63, 2, 0), (8, 0, 4)):
        buf = randn(g, 50 * (width + pad) + shift, dtype=dtype)
        table = buf.as_strided((50, width), (width + pad, 1), shift)
        assert torch.equal(rs.embedding(table, ids, 3.0), lookup(table, ids, 3.0))
        out = torch.full((60, width + 5), 9.0, dtype=dtype, device="cuda")
        rs.embedding(table, ids.reshape(-1), 3.0, out=out[:, 2:2 + width])
        assert torch.equal(out[:, 2:2 + width], lookup(table, ids.reshape(-1), 3.0))
        assert (out[:, :2] == 9).all() and (out[:, 2 + width:] == 9).all()
    whole = torch.empty(3, 4, 5, 8, dtype=dtype, device="cuda")
    assert rs.embedding(table, ids, out=whole) is whole and torch.equal(whole, lookup(table, ids, 1.0))
    table[3] = math.inf  # a padded token beside an infinite row is 0 all the same
    assert (rs.embedding(table, torch.tensor([-1], device="cuda")) == 0).all()


def check_grad(rs, up, ids, vocab, scale=1.0, padding_id=-1, dtype=None):
    """All three forms; returns the table."""
    dtype = dtype or up.dtype
    width = up.shape[-1]
    kw = {"scale": scale, "padding_id": padding_id}
    want, size, n = vo.embedding_grad(up, ids, vocab, scale, padding_id)
    bound = vo.embedding_bound(want, size, n, dtype)
    table = rs.embedding_grad(up, ids, vocab, dtype=dtype, **kw)
    assert table.dtype is dtype and table.shape == (vocab, width)
    within(table, want, bound, "table")
    assert (table[n == 0] == 0).all()

    before = torch.randn(vocab, width, device="cuda").to(dtype)
    sums = rs.embedding_grad(up, ids, vocab, grad_out=before.clone(), accumulate=True, **kw)
    total = before.double() + want
    u = vo.ROUND[dtype][0]
    within(sums, total, bound + (total.abs() * 1.01 + before.double().abs() * 2.0 ** -23) * max(u, 2.0 ** -23), "sum")
    assert torch.equal(sums[n == 0], before[n == 0])

    room = min(ids.numel(), vocab)
    rows_out = torch.full((room, width), 7.0, dtype=dtype, device="cuda")
    row_ids, rows, count = rs.embedding_grad_rows(up, ids, vocab, rows_out=rows_out, **kw)
    named = (n > 0).nonzero()[:, 0]
    assert count.dtype is torch.int32 and int(count) == named.numel()
    c = named.numel()
    assert torch.equal(row_ids[:c], named) and (row_ids[c:] == -1).all()
    assert torch.equal(rows[:c], table[named])
    assert (rows[c:] == 7).all()  # left as they were
    return table


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", WIDTHS)
def test_gradient_widths(rs, width, dtype):
    g = gen(width)
    for n in (1, 2, 31, 33, 500):
        ids = ids_of(g, n, 203)
        check_grad(rs, randn(g, n, width, dtype=dtype), ids, 203, math.sqrt(width))


@pytest.mark.parametrize("dtype,out", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                       (torch.float16, torch.float16), (torch.float16, torch.float32),
                                       (torch.float32, torch.float32)])
@pytest.mark.parametrize("n,vocab,width", [(3000, 1000, 64), (5000, 40000, 33), (9001, 131072, 40),
                                           (20000, 300, 256), (100003, 50001, 16), (300000, 1000, 8)])
def test_gradient_sizes(rs, n, vocab, width, dtype, out):
    g = gen(n)
    ids = ids_of(g, n, vocab)
    check_grad(rs, randn(g, n, width, dtype=dtype), ids, vocab, 1.0, dtype=out)


@pytest.mark.parametrize("n", [1, 31, 32, 33, 64, 127, 128, 129, 255, 256, 257, 1000, 2048, 2049, 4096,
                               4097, 5000, 8193, 40000])
def test_gradient_of_one_id(rs, n):
    """Every token the same: one run, of pieces that end anywhere."""
    g = gen(n)
    up = randn(g, n, 40)
    check_grad(rs, up, torch.full((n,), 17, device="cuda"), 90)
    mixed = torch.full((n,), 17, device="cuda")
    mixed[:n // 3] = 5
    mixed[n // 2::50] = 63
    check_grad(rs, up, mixed, 90)


@pytest.mark.parametrize("n", [1000, 2048, 5000, 20000])
@pytest.mark.parametrize("ids_named", [3, 20, 60, 100])
def test_gradient_of_many_long_runs(rs, n, ids_named):
    """Runs of more than a warp's tokens in wide rows: each run's columns are
    shared by many warps, which have to agree on who adds up what."""
    g = gen(n + ids_named)
    ids = torch.randperm(5000, generator=g, device="cuda")[:ids_named][ids_of(g, n, ids_named, "all")]
    check_grad(rs, randn(g, n, 2056, dtype=torch.bfloat16), ids, 5000, dtype=torch.float32)
    check_grad(rs, randn(g, n, 515), ids, 5000)
    check_grad(rs, randn(g, n, 3001, dtype=torch.float16), ids, 5000)  # element by element


@pytest.mark.parametrize("n,width,dtype", [(70001, 2056, torch.bfloat16), (70001, 515, torch.float32),
                                           (80003, 3001, torch.float16), (131073, 1024, torch.bfloat16),
                                           (66000, 40, torch.float16)])
@pytest.mark.parametrize("ids_named", [3, 60, 3000])
def test_gradient_of_many_tokens_in_wide_rows(rs, ids_named, n, width, dtype):
    """More tokens than one cluster sorts, in rows that many warps share: long
    runs of each, of a third of all and of some, and short ones."""
    g = gen(n + ids_named)
    ids = torch.randperm(5000, generator=g, device="cuda")[:ids_named][ids_of(g, n, ids_named, "all")]
    ids[: n // 3] = ids[-1]
    ids[1::1000] = -1
    check_grad(rs, randn(g, n, width, dtype=dtype), ids, 5000, dtype=torch.float32)


@pytest.mark.parametrize("n", [700, 6000])
def test_gradient_of_dropped_and_padded_tokens(rs, n):
    g = gen(3)
    up = randn(g, n, 72, dtype=torch.bfloat16)
    ids = ids_of(g, n, 500)
    ids[::4] = -1
    ids[1::9] = 500
    ids[2::9] = 2 ** 40
    check_grad(rs, up, ids, 500, 2.0, padding_id=0)
    check_grad(rs, up, ids.clamp(-1, 1000).int(), 500, 2.0, padding_id=499)
    up[::4] = math.nan  # what is dropped is not added
    check_grad(rs, up, ids, 500)
    check_grad(rs, up, torch.full((n,), -1, device="cuda"), 500)
    check_grad(rs, up, torch.full((n,), 7, device="cuda"), 500, padding_id=7)


def test_gradient_of_no_tokens_and_one_row(rs):
    up = torch.empty(0, 24, device="cuda")
    check_grad(rs, up, torch.empty(0, dtype=torch.int64, device="cuda"), 100)
    g = gen(4)
    check_grad(rs, randn(g, 300, 24), torch.zeros(300, dtype=torch.int64, device="cuda"), 1)
    check_grad(rs, randn(g, 5000, 24), torch.zeros(5000, dtype=torch.int64, device="cuda"), 1)


@pytest.mark.parametrize("n", [400, 7000])
@pytest.mark.parametrize("dtype", TYPES)
def test_gradient_strides_shapes_and_alignments(rs, dtype, n):
    g = gen(5)
    ids = ids_of(g, n, 200)
    for width, pad, shift in ((64, 8, 8), (64, 2, 2), (64, 1, 1), (63, 2, 0), (8, 0, 4)):
        buf = torch.full((n * (width + pad) + shift,), math.nan, dtype=dtype, device="cuda")
        up = buf.as_strided((n, width), (width + pad, 1), shift)
        up.copy_(randn(g, n, width))
        table = check_grad(rs, up, ids, 200)
        out = torch.full((200, width + 5), 9.0, dtype=dtype, device="cuda")
        rs.embedding_grad(up, ids, 200, grad_out=out[:, 2:2 + width])
        assert torch.equal(out[:, 2:2 + width], table)
        assert (out[:, :2] == 9).all() and (out[:, 2 + width:] == 9).all()
    # outputs that begin 16 bytes into a line, of either type
    up = randn(g, n, 64, dtype=dtype)
    for out_type in {dtype, torch.float32}:
        first = 16 // torch.empty(0, dtype=out_type).element_size()
        buf = torch.full((200 * 64 + 2 * first,), 9.0, dtype=out_type, device="cuda")
        out = buf[first:first + 200 * 64].view(200, 64)
        rs.embedding_grad(up, ids, 200, grad_out=out)
        assert torch.equal(out, rs.embedding_grad(up, ids, 200, dtype=out_type))
        assert (buf[:first] == 9).all() and (buf[first + 200 * 64:] == 9).all()
        table = buf[first:first + 200 * 64].view(200, 64)
        assert torch.equal(rs.embedding(table, ids, 2.0), lookup(table, ids, 2.0))
    up = randn(g, 4, n // 4, 16, dtype=dtype)
    check_grad(rs, up, ids[:4 * (n // 4)].reshape(4, n // 4), 200)


def test_gradient_in_a_large_vocabulary(rs):
    g = gen(6)
    for vocab in (255, 256, 65535, 65536, 1 << 20, (1 << 24) + 3):
        n = 6000
        ids = ids_of(g, n, vocab, "all")
        ids[0], ids[1] = vocab - 1, 0
        check_grad(rs, randn(g, n, 4), ids, vocab)
        check_grad(rs, randn(g, 300, 4), ids[:300].contiguous(), vocab)


def test_offsets_beyond_32_bits(rs):
    """A table of more than 2^32 bytes and 2^31 elements."""
    vocab, width = 70000, 32768
    g = gen(7)
    table = torch.zeros(vocab, width, dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([0, vocab - 1, 66000, 65536, vocab - 1, 3], device="cuda")
    table[ids] = randn(g, 6, width, dtype=torch.bfloat16)
    assert torch.equal(rs.embedding(table, ids), table[ids])
    up = randn(g, 6, width, dtype=torch.bfloat16)
    out = rs.embedding_grad(up, ids, vocab, grad_out=table)
    want, size, n = vo.embedding_grad(up, torch.tensor([0, 4, 2, 1, 4, 3], device="cuda"), 5)
    at = torch.tensor([0, 65536, 66000, 3, vocab - 1], device="cuda")
    within(out[at], want, vo.embedding_bound(want, size, n, torch.bfloat16), "rows")
    out[at] = 0
    assert not out.any()


def test_same_bits_in_every_run(rs):
    g = gen(8)
    for n in (600, 30000):
        up, ids = randn(g, n, 256, dtype=torch.bfloat16), ids_of(g, n, 100)
        want = rs.embedding_grad(up, ids, 100)
        for _ in range(10):
            assert torch.equal(rs.embedding_grad(up, ids, 100), want)


def test_autograd_and_differences(rs):
    g = gen(9)
    table = randn(g, 40, 12)
    ids = ids_of(g, 30, 40).reshape(5, 6)
    ids[0, 0], ids[1, 1] = -1, 39
    leaf = table.clone().requires_grad_(True)
    out = rs.embedding(leaf, ids, 3.0, padding_id=39)
    assert torch.equal(out, lookup(table, ids, 3.0))
    up = randn(g, 5, 6, 12)
    (out * up).sum().backward()
    want, size, n = vo.embedding_grad(up, ids, 40, 3.0, 39)
    within(leaf.grad, want, vo.embedding_bound(want, size, n, torch.float32), "autograd")
    # the lookup is linear: a difference of steps of 1 is the gradient, but for rounding
    i, j = int(ids[2, 2]), 5
    step = torch.zeros_like(table)
    step[i, j] = 1.0
    value = lambda t: (rs.embedding(t, ids, 3.0).double() * up).sum()  # noqa: E731
    slope = value(table + step) - value(table)
    assert abs(float(slope - want[i, j])) <= 2.0 ** -22 * float(size[i, j] + 3 * up[ids == i][:, j].abs().sum() * 5)
    rs.embedding(leaf, ids).sum().backward()  # an upstream gradient that is one number
    leaf.grad = None
    rs.embedding(leaf, ids).sum().backward()
    want, _, _ = vo.embedding_grad(torch.ones(5, 6, 12, device="cuda"), ids, 40)
    assert torch.equal(leaf.grad.double(), want)


def test_streams_and_both_at_once(rs):
    g = gen(10)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    up, ids = randn(g, 9000, 128, dtype=torch.bfloat16), ids_of(g, 9000, 3000)
    vp, jds = randn(g, 700, 64), ids_of(g, 700, 500)
    want = rs.embedding_grad(up, ids, 3000), rs.embedding_grad(vp, jds, 500)
    torch.cuda.synchronize()
    for _ in range(20):
        got = (rs.embedding_grad(up, ids, 3000, stream=a), rs.embedding_grad(vp, jds, 500, stream=b))
        a.synchronize(), b.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("n", [500, 9000])
def test_graph_replays_on_new_tokens(rs, n):
    g = gen(11)
    table = randn(g, 2000, 64, dtype=torch.bfloat16)
    ids = ids_of(g, n, 2000)
    up = randn(g, n, 64, dtype=torch.bfloat16)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        rs.embedding_grad(up, ids, 2000)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = rs.embedding(table, ids, 8.0)
        whole = rs.embedding_grad(up, ids, 2000)
        row_ids, rows, count = rs.embedding_grad_rows(up, ids, 2000)
    for _ in range(3):
        ids.copy_(ids_of(g, n, 2000))
        up.copy_(randn(g, n, 64))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, lookup(table, ids, 8.0))
        want = rs.embedding_grad(up, ids, 2000)
        assert torch.equal(whole, want)
        c = int(count)
        assert torch.equal(rows[:c], want[row_ids[:c]])


def test_temp_is_the_callers(rs):
    g = gen(12)
    for n in (100, 5000):
        up, ids = randn(g, n, 32), ids_of(g, n, 400)
        temp = torch.full((rs.embedding_grad_temp_bytes(n, 400, 32),), 0xAA, dtype=torch.uint8, device="cuda")
        want = rs.embedding_grad(up, ids, 400)
        for _ in range(2):
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            assert torch.equal(rs.embedding_grad(up, ids, 400, temp=temp, status_out=status), want)
            assert int(status) == 0
        with pytest.raises(rs.RadixSortError):
            rs.embedding_grad(up, ids, 400, temp=temp[:-256])


class FailedSort:
    """The sort inside a call on `temp` fails: while the call runs, the word that
    its tiles say so by, the first of the sort's part of the scratch, is written
    again and again from another stream."""

    def __init__(self, rs, temp, n, vocab):
        sort = -(-rs.temp_bytes(n, 4, 4, 0, vocab.bit_length(), 8) // 256) * 256
        self.word = temp[temp.numel() - sort:][:4].view(torch.int32)
        self.stream = torch.cuda.Stream()
        self.stream.wait_stream(torch.cuda.current_stream())
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph, stream=self.stream):
            for _ in range(1000):
                self.word.fill_(4)
        self.graph.replay()
        torch.cuda.synchronize()

    def __call__(self, call):
        torch.cuda._sleep(20_000_000)  # all is queued before any of it begins
        begin = torch.cuda.current_stream().record_event()
        torch.cuda._sleep(100_000)     # the word's writer first
        self.stream.wait_event(begin)
        with torch.cuda.stream(self.stream):
            self.graph.replay()
        got = call()
        torch.cuda.synchronize()
        return got


@pytest.mark.parametrize("n,vocab,dtype", [(100_000, 5000, torch.bfloat16), (300_000, 200, torch.float32)])
def test_a_sort_that_fails(rs, n, vocab, dtype):
    """A whole table is NaN, one that is added to stays as it was, there are no
    rows, and the status says so; the next call on the same scratch is right."""
    g = gen(13)
    width = 24
    up, ids = randn(g, n, width, dtype=dtype), ids_of(g, n, vocab)
    before = randn(g, vocab, width)
    temp = torch.empty(rs.embedding_grad_temp_bytes(n, vocab, width), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    table, sums = (torch.full((vocab, width), 7.0, device="cuda", dtype=t) for t in (dtype, torch.float32))
    sums.copy_(before)
    row_ids = torch.full((vocab,), 7, dtype=torch.int64, device="cuda")
    rows, count = torch.full((vocab, width), 7.0, device="cuda", dtype=dtype), status + 7
    kw = {"temp": temp, "status_out": status}

    def whole():
        return rs.embedding_grad(up, ids, vocab, grad_out=table, **kw)

    def added():
        return rs.embedding_grad(up, ids, vocab, grad_out=sums, accumulate=True, **kw)

    def named():
        return rs.embedding_grad_rows(up, ids, vocab, row_ids_out=row_ids, rows_out=rows, count_out=count, **kw)

    fails = FailedSort(rs, temp, n, vocab)
    for call in (whole, added, named):
        call()  # (kernels are loaded, which waits for all streams)
        assert int(status) == 0 and int(fails.word) == 0
    for out in (table, rows, row_ids, count):
        out.fill_(7)
    sums.copy_(before)
    for call in (whole, added, named):
        status.zero_()
        fails(call)
        assert int(status) == rs.RS_ERR_LOOKBACK_TIMEOUT
    assert table.isnan().all()
    assert torch.equal(sums, before)
    assert int(count) == 0 and (row_ids == -1).all() and (rows == 7).all()
    fails(lambda: rs.embedding_grad(up, ids, vocab, grad_out=table, temp=temp))  # nobody asks
    assert table.isnan().all()
    status.zero_()
    want, size, terms = vo.embedding_grad(up, ids, vocab)
    within(whole(), want, vo.embedding_bound(want, size, terms, dtype), "the next call")
    named()
    c = int(count)
    assert torch.equal(rows[:c], table[row_ids[:c]]) and int(status) == 0
