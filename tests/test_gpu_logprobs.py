"""Log probabilities of tokens, entropy and top alternatives against their
formulas in 64 bits: types, odd and long rows, strides and alignments, ties in
every number, masks, -inf and NaN, long lists, streams, graphs; the gradient
against its formula and against differences."""
import math

import pytest
import torch

from tests import vocab_oracle as vo
from tests.loss_bounds import within

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]


def rows_of(rows, cols, dtype, seed, pad=0, shift=0, spread=3.0):
    """Scores as a view with padded rows that starts `shift` elements into its
    buffer; the padding holds NaN."""
    g = torch.Generator("cuda").manual_seed(seed)
    buf = torch.full((rows * (cols + pad) + shift,), math.nan, dtype=dtype, device="cuda")
    x = buf[shift:].as_strided((rows, cols), (cols + pad, 1), shift)
    x.copy_((torch.randn(rows, cols, generator=g, device="cuda") * spread).to(dtype))
    return x, g


def tokens_of(x, k, g):
    return torch.randint(0, x.shape[1], (x.shape[0], k), generator=g, device="cuda")


def check(rs, x, tokens=None, top=0, tau=1.0):
    want = vo.Logprobs(x, tau)
    got = rs.token_logprobs(x, tokens, top, tau)
    within(got.entropy, want.entropy, want.entropy_error, "entropy")
    within(got.lse, want.lse, want.lse_error, "lse")
    within(got.stats[:, 0], want.m, torch.zeros_like(want.m), "largest score")
    within(got.stats[:, 1], want.log_sum, want.stats_error, "log-sum")
    if tokens is None:
        assert got.logprobs is None
    else:
        logp, bound = want.logprobs(tokens.reshape(x.shape[0], -1))
        within(got.logprobs.reshape(logp.shape), logp, bound, "logprobs")
    if top:
        columns = want.top(top)
        assert got.top_ids.dtype is torch.int64 and torch.equal(got.top_ids, columns)
        logp, bound = want.logprobs(columns)
        logp = torch.where(columns < 0, torch.full_like(logp, -math.inf), logp)
        within(got.top_logprobs, logp, bound, "top logprobs")
    else:
        assert got.top_ids is None and got.top_logprobs is None
    return got, want


WIDTHS = [(1, 1), (3, 2), (2, 7), (5, 8), (3, 31), (4, 33), (3, 255), (2, 1000), (3, 4097),
          (2, 8191), (2, 16384), (2, 50001), (1, 65536), (2, 131075), (1, 300007)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", WIDTHS)
def test_widths(rs, rows, cols, dtype):
    x, g = rows_of(rows, cols, dtype, rows + cols)
    for top, k in ((0, 1), (1, 0), (5, 3), (33, 1), (100, 2)):
        check(rs, x, tokens_of(x, k, g) if k else None, top)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,shift", [(1, 0), (0, 1), (3, 5), (64, 8), (7, 7)])
def test_strides_and_alignments(rs, dtype, pad, shift):
    for cols in (1003, 20001):
        x, g = rows_of(5, cols, dtype, pad + shift, pad, shift)
        check(rs, x, tokens_of(x, 2, g), 20)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(700, 3000), (1500, 900), (1000, 33000), (160, 131072)])
def test_many_rows(rs, rows, cols, dtype):
    x, g = rows_of(rows, cols, dtype, 3)
    check(rs, x, tokens_of(x, 1, g), 20, 0.7)


@pytest.mark.parametrize("dtype,cols", [(torch.bfloat16, 5000003), (torch.float32, 3000001)])
def test_rows_beyond_a_slot_per_batch(rs, dtype, cols):
    x, g = rows_of(1, cols, dtype, 4)
    check(rs, x, tokens_of(x, 1, g), 64)
    x[0, :cols // 2] = 50.0  # a long tie
    check(rs, x, tokens_of(x, 1, g), 9)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,top", [(3, 1024, 1024), (2, 50001, 1024), (5, 700, 1000),
                                           (300, 20000, 129), (2, 200000, 512), (1, 131072, 256)])
def test_long_lists(rs, rows, cols, top, dtype):
    x, g = rows_of(rows, cols, dtype, top)
    check(rs, x, tokens_of(x, 1, g), top)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,top", [(4100, 600, 100), (4500, 2000, 128), (4100, 2000, 40),
                                           (300, 2000, 300), (300, 2048, 700), (40, 1500, 129),
                                           (20, 9000, 1024)])
def test_long_lists_of_short_rows(rs, rows, cols, top, dtype):
    """Nearly all of a row's scores are candidates, and more than are put in
    order at once."""
    x, g = rows_of(rows, cols, dtype, top)
    check(rs, x, None, top)
    tied = torch.randint(0, 5, x.shape, generator=g, device="cuda").to(dtype)
    check(rs, tied, None, top)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(4, 300), (3, 20000), (2, 131072), (600, 9000)])
def test_ties_go_to_the_lower_column(rs, rows, cols, dtype):
    x, g = rows_of(rows, cols, dtype, 7)
    t = tokens_of(x, 1, g)
    for values in (1, 2, 5, 40):  # so many different scores
        tied = torch.randint(0, values, x.shape, generator=g, device="cuda").to(dtype)
        for top in (1, 20, 64, 200):
            check(rs, tied, t, top)
    zeros = torch.where(torch.rand(x.shape, generator=g, device="cuda") < 0.5, 0.0, -0.0).to(dtype)
    check(rs, zeros, t, 20)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,shift", [(3, 5003, 3), (4200, 3000, 0), (2, 200001, 0)])
def test_long_ties_below_a_few_better_ones(rs, rows, cols, shift, dtype):
    """More equal scores than fit beside others that are better, positive and
    negative, the first of them early, late, or one in a hundred."""
    x, g = rows_of(rows, cols, dtype, 21, shift % 2, shift)
    for value in (1.0, -3.0, 0.0):
        x.fill_(value)
        x[:, 7::1000] = value + 0.5
        x[:, cols - 3] = 9.0
        check(rs, x, None, 60)
        x[:, :cols // 2] = -20.0     # ties from the middle on
        check(rs, x, None, 100)
        check(rs, x, None, 300)
        x.fill_(-20.0)
        x[:, ::100] = value
        check(rs, x, None, min(20, cols // 200))


@pytest.mark.parametrize("dtype", TYPES)
def test_orders_that_gather_the_best_in_one_place(rs, dtype):
    for cols in (5000, 70000):
        x, g = rows_of(6, cols, dtype, 8)
        ordered = torch.sort(x.float(), dim=1).values.to(dtype)
        for top in (20, 64, 128):
            check(rs, ordered, tokens_of(x, 1, g), top)
            check(rs, ordered.flip(1).contiguous(), tokens_of(x, 1, g), top)
        x[:, 64:128] = 40.0 + x[:, 64:128]  # eight neighbouring vectors hold them all
        check(rs, x, tokens_of(x, 1, g), 40)


@pytest.mark.parametrize("dtype", TYPES)
def test_masks(rs, dtype):
    low = torch.finfo(dtype).min
    for cols in (70, 9001, 70000):
        x, g = rows_of(9, cols, dtype, 9)
        x[0] = -math.inf                      # nothing at all
        x[1, 1:] = -math.inf                  # one score
        x[2, :-3] = -math.inf                 # three at the end
        x[3] = low                            # the lowest value, everywhere
        x[4, 5:] = low                        # and beside others
        x[5, ::2] = -math.inf
        x[6] = 6.0e4                          # large ones, all alike
        x[7, :3] = torch.tensor([low, -math.inf, 0.0], dtype=dtype)
        got, _ = check(rs, x, tokens_of(x, 3, g), 20)
        assert got.entropy[0] == 0 and got.lse[0] == -math.inf
        assert (got.top_ids[1, 1:] == -1).all() and got.top_ids[1, 0] == 0
        # One score x: its exponent, x log2 e less its own rounding to o, is off
        # by |o| 2^-24 at most; the entropy's terms e y and e (o's rounding)
        # cancel but for a rounding of theirs, 2^-24 of that again.
        assert abs(got.entropy[1]) <= 2.0 ** -48 * 1.5 * (abs(float(x[1, 0])) + 1)
        assert got.top_logprobs[1, 0] == 0


def test_large_scores_and_temperatures(rs):
    for dtype in (torch.bfloat16, torch.float32):
        x, g = rows_of(6, 5000, dtype, 10)
        x[0] += 1e4
        x[1] -= 1e6
        x[2] = -1e30
        x[2, 7] = -1e29
        x[3, 100:] = 3e38
        x[4, 100:] = -3e38
        t = tokens_of(x, 2, g)
        for tau in (1.0, 0.01, 50.0, 1e10, 1e-10):
            got = rs.token_logprobs(x, t, 8, tau)
            want = vo.Logprobs(x, tau)
            assert torch.equal(got.top_ids, want.top(8))
            within(got.stats[:, 1], want.log_sum, want.stats_error, f"log-sum at {tau}")
            within(got.entropy, want.entropy, want.entropy_error, f"entropy at {tau}")
            logp, bound = want.logprobs(t)
            held = logp.abs() < 3e38  # what a float holds
            within(torch.where(held, got.logprobs.double(), logp), logp, bound, f"logprobs at {tau}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(8, 64), (8, 3000), (300, 12000), (8, 40000), (8, 400003)])
def test_scores_further_apart_than_a_float(rs, rows, cols, dtype):
    """Scores of both signs at the type's limits, at temperatures that make
    their difference a small one; the larger ones early, late, and anywhere."""
    for tau in (1e36, 1e37, 8e37, 3.3e38):
        x, g = rows_of(rows, cols, dtype, 26)
        x[0::4, :cols // 2], x[0::4, cols // 2:] = -3.3e38, 3.3e38
        x[1::4], x[1::4, cols - 1] = -3.3e38, 3.3e38
        x[2::4] = ((torch.rand(rows // 4, cols, generator=g, device="cuda") * 2 - 1) * 3.3e38).to(dtype)
        x[3::4, :cols // 2] = -3.3e38
        t = tokens_of(x, 2, g)
        t[:, 0] = cols - 1
        check(rs, x, t, 20, tau)
        if tau < 2.0 ** 126:  # (above, 1 / tau has fewer than 24 bits)
            check_grad(rs, x, g, tokens=t, top=3, tau=tau)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("cols", [50, 40000])
def test_nan_and_infinity_stay_in_their_rows(rs, dtype, cols):
    x, g = rows_of(8, cols, dtype, 11)
    clean = x.clone()
    x[1, cols // 2] = math.nan
    x[3, cols - 1] = math.inf
    x[5] = math.nan
    x[6, ::3] = -math.nan
    t = tokens_of(x, 2, g)
    got = rs.token_logprobs(x, t, 6)
    bad = torch.tensor([1, 3, 5, 6], device="cuda")
    for name in ("logprobs", "entropy", "top_logprobs", "lse", "stats"):
        part = getattr(got, name)[bad]
        assert part.isnan().flatten(1).any(1).all() if part.dim() > 1 else part.isnan().all(), name
    assert got.logprobs[bad].isnan().all() and got.top_logprobs[bad].isnan().all()
    assert (got.top_ids[bad] == -1).all()
    want = rs.token_logprobs(clean, t, 6)
    good = torch.tensor([0, 2, 4, 7], device="cuda")
    for a, b in zip(got, want):
        assert torch.equal(a[good], b[good])
    up = torch.ones(8, device="cuda")
    grad = rs.token_logprobs_backward(x, got.stats, got.entropy, t, None, torch.ones(8, 2, device="cuda"), up)
    assert grad[bad].isnan().all() and not grad[good].isnan().any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(4, 65536), (4, 20001), (4200, 3000)])
def test_nan_beside_long_ties(rs, rows, cols, dtype):
    """Rows of more equal scores than fit among the candidates, with NaN in a few
    columns, in thousands, and in nearly all: values NaN, ids -1, whatever the
    ties' sign; rows without NaN between them are not touched by it."""
    x, g = rows_of(rows, cols, dtype, 25)
    t = tokens_of(x, 1, g)
    draw = torch.rand(rows, cols, generator=g, device="cuda")
    for value in (1.0, 0.0, -3.0, torch.finfo(dtype).min):
        for better in (False, True):
            x.fill_(value)
            if better:
                x[:, 7::50] = value + 0.5 if value > -1e4 else 0.0
            clean = x.clone()
            for share in (0.001, 0.3, 0.99):
                gone = draw < share
                gone[:, 0] = True
                gone[1::4] = False
                x.copy_(torch.where(gone, torch.full_like(x, math.nan), clean))
                for top in (20, 128, 300):
                    got = rs.token_logprobs(x, t, top)
                    want = rs.token_logprobs(clean[1::4], t[1::4], top)
                    bad = gone[:, 0]
                    for name in ("logprobs", "entropy", "lse", "top_logprobs"):
                        assert getattr(got, name)[bad].isnan().all(), name
                    assert (got.top_ids[bad] == -1).all()
                    assert all(torch.equal(a[1::4], b) for a, b in zip(got, want))


def test_tokens_outside_and_repeated_and_many(rs):
    x, g = rows_of(7, 3001, torch.bfloat16, 12)
    t = tokens_of(x, 6, g)
    t[0, 0], t[1, 1], t[2, 2], t[3] = -1, 3001, 2 ** 40, -1
    t[4, :] = t[4, 0]
    check(rs, x, t, 3)
    short = tokens_of(x, 4, g).int()
    check(rs, x, short, 0)
    check(rs, x, tokens_of(x, 1, g)[:, 0].contiguous(), 4)     # one per row, as a vector
    check(rs, x, tokens_of(x, 9, g)[:, 2:7], 4)                # padded rows of tokens
    check(rs, x, tokens_of(x, 1024, g), 0)
    check(rs, x, torch.empty(7, 0, dtype=torch.int64, device="cuda"), 2)


def test_no_rows(rs):
    x = torch.empty(0, 100, device="cuda")
    got = rs.token_logprobs(x, torch.empty(0, 2, dtype=torch.int64, device="cuda"), 5)
    assert got.logprobs.shape == (0, 2) and got.top_ids.shape == (0, 5)
    assert rs.token_logprobs_backward(x, got.stats).shape == (0, 100)


# -------------------------------------------------------------------- gradient
def check_grad(rs, x, g, k=1, top=0, entropy=True, lse=True, tau=1.0, grad_out=None, tokens=None):
    rows = x.shape[0]
    want = vo.Logprobs(x, tau)
    tokens = tokens_of(x, k, g) if tokens is None and k else tokens
    fwd = rs.token_logprobs(x, tokens, top, tau)

    def up(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    gl, gt = up(*tokens.shape) if tokens is not None else None, up(rows, top) if top else None
    gh, gs = up(rows) if entropy else None, up(rows) if lse else None
    entries = [(tokens.reshape(rows, -1), gl.reshape(rows, -1))] if tokens is not None else []
    entries += [(fwd.top_ids, gt)] if top else []
    grad, bound = want.grad(entries, gh, gs)
    got = rs.token_logprobs_backward(x, fwd.stats, fwd.entropy, tokens, fwd.top_ids, gl, gh, gs, gt,
                                     tau, grad_out=grad_out)
    within(got, grad, bound, "gradient")
    return got


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", WIDTHS)
def test_gradient_widths(rs, rows, cols, dtype):
    x, g = rows_of(rows, cols, dtype, rows + cols)
    check_grad(rs, x, g)
    check_grad(rs, x, g, k=3, top=min(cols, 20), tau=0.7)
    check_grad(rs, x, g, k=0, top=5, entropy=False, lse=False)
    check_grad(rs, x, g, k=0, entropy=True, lse=False, tau=2.0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,shift", [(1, 0), (0, 1), (3, 5), (64, 8), (7, 7)])
def test_gradient_strides_and_alignments(rs, dtype, pad, shift):
    for cols in (1003, 20001):
        x, g = rows_of(5, cols, dtype, pad + shift, pad, shift)
        check_grad(rs, x, g, k=2, top=4)
        out = torch.full((5, cols + 3), 7.0, dtype=dtype, device="cuda")
        check_grad(rs, x, g, k=2, top=4, grad_out=out[:, 1:1 + cols])
        assert (out[:, 0] == 7).all() and (out[:, 1 + cols:] == 7).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(1, 100000), (40, 131072), (3, 500), (900, 9000)])
def test_gradient_in_place(rs, rows, cols, dtype):
    x, g = rows_of(rows, cols, dtype, 13)
    copy = x.clone()
    state = g.get_state()
    want = check_grad(rs, copy, g, k=3, top=10)
    g.set_state(state)
    over = x.clone()
    fwd = rs.token_logprobs(over, tokens_of(over, 3, g), 10)
    g.set_state(state)
    t = tokens_of(over, 3, g)
    gl, gt = (torch.randn(*t.shape, generator=g, device="cuda"),
              torch.randn(rows, 10, generator=g, device="cuda"))
    gh, gs = torch.randn(rows, generator=g, device="cuda"), torch.randn(rows, generator=g, device="cuda")
    got = rs.token_logprobs_backward(over, fwd.stats, fwd.entropy, t, fwd.top_ids, gl, gh, gs, gt,
                                     grad_out=over)
    assert got.data_ptr() == over.data_ptr() and torch.equal(got, want)


def test_gradient_masks_and_repeats(rs):
    for dtype in TYPES:
        low = torch.finfo(dtype).min
        x, g = rows_of(7, 9001, dtype, 14)
        x[0] = -math.inf
        x[1, 1:] = -math.inf
        x[2, ::2] = -math.inf
        x[3] = low
        x[4, 5:] = low
        t = tokens_of(x, 40, g)
        t[:, :20] = t[:, :1]  # one column twenty times
        t[5] = -1
        grad = check_grad(rs, x, g, tokens=t, top=12)
        assert (grad[0] == 0).all()
        only = rs.token_logprobs_backward(x, rs.token_logprobs(x).stats, tokens=t,
                                          grad_logprobs=torch.ones_like(t, dtype=torch.float32))
        assert (only[5] == 0).all()  # no token, no gradient


def test_gradient_of_long_lists(rs):
    x, g = rows_of(3, 5000, torch.float32, 15)
    check_grad(rs, x, g, k=1024, top=1024)


@pytest.mark.parametrize("rows,cols", [(2, 900), (5, 60000), (500, 3001)])
def test_gradient_of_long_lists_that_repeat(rs, rows, cols):
    x, g = rows_of(rows, cols, torch.bfloat16, 18)
    for k, top in ((64, 0), (65, 0), (200, 130), (1024, 100)):
        t = torch.randint(0, 40, (rows, k), generator=g, device="cuda")
        t[0] = 7                # one column alone
        t[1, ::3] = -1
        t[1, 1::3] = cols       # outside as well
        check_grad(rs, x, g, tokens=t, top=top)
        again = [rs.token_logprobs_backward(x, rs.token_logprobs(x).stats, tokens=t,
                                            grad_logprobs=torch.ones(rows, k, device="cuda") / 3)
                 for _ in range(2)]
        assert torch.equal(*again)


def test_gradient_is_that_of_differences(rs):
    """d/dx by central differences of the forward call's own results, in rows
    of few scores.  A difference of 2 h of values with error e is off by e / h
    and by h^2 / 6 times a third derivative, at most 8 here."""
    g = torch.Generator("cuda").manual_seed(16)
    x = torch.randn(4, 6, generator=g, device="cuda")
    t = torch.tensor([[0, 3], [5, 5], [2, -1], [1, 4]], device="cuda")
    gl, gh, gs = (torch.randn(4, 2, generator=g, device="cuda"), torch.randn(4, generator=g, device="cuda"),
                  torch.randn(4, generator=g, device="cuda"))
    gt = torch.randn(4, 2, generator=g, device="cuda")

    def value(x):
        f = rs.token_logprobs(x, t, 2, 0.8)
        live = (t >= 0).double()
        return ((f.logprobs.double() * gl * live).sum(1) + f.entropy.double() * gh + f.lse.double() * gs
                + (f.top_logprobs.double() * gt).sum(1))

    f = rs.token_logprobs(x, t, 2, 0.8)
    got = rs.token_logprobs_backward(x, f.stats, f.entropy, t, f.top_ids, gl, gh, gs, gt, 0.8)
    h = 2.0 ** -6
    size = 4 + gl.abs().sum(1) + gh.abs() + gs.abs() + gt.abs().sum(1)
    for j in range(6):
        step = torch.zeros_like(x)
        step[:, j] = h
        slope = (value(x + step) - value(x - step)) / (2 * h)
        bound = size.double() * (64 * 2.0 ** -24 / h + 8 / 0.8 ** 3 * h * h)
        within(got[:, j], slope, bound, f"slope {j}")


def test_autograd(rs):
    x, g = rows_of(5, 2000, torch.float32, 17)
    t = tokens_of(x, 2, g)
    leaf = x.clone().requires_grad_(True)
    out = rs.token_logprobs(leaf, t, 3, 0.9)
    assert not out.top_ids.requires_grad and not out.stats.requires_grad
    (out.logprobs.sum() - 0.1 * out.entropy.sum() + (out.lse ** 2).sum() + out.top_logprobs[:, 0].sum()).backward()
    z = x.double().requires_grad_(True)
    logq = torch.log_softmax(z / float(torch.tensor(0.9)), 1)
    lse = torch.logsumexp(z / float(torch.tensor(0.9)), 1)
    (logq.gather(1, t).sum() + 0.1 * (logq.exp() * logq).sum() + (lse ** 2).sum() + logq.amax(1).sum()).backward()
    want = vo.Logprobs(x, 0.9)
    one = torch.zeros(5, 3, device="cuda")
    one[:, 0] = 1
    _, bound = want.grad([(t, torch.ones(5, 2, device="cuda")), (out.top_ids, one)],
                         torch.full((5,), -0.1, device="cuda"), 2 * want.lse)
    lse_part = want.q * 2 * want.lse_error[:, None] / 0.9
    within(leaf.grad, z.grad, bound + lse_part, "autograd")
    with torch.no_grad():
        assert not rs.token_logprobs(leaf, t).logprobs.requires_grad
    alone = rs.token_logprobs(leaf, t, 0, 0.9)
    grad, = torch.autograd.grad(alone.entropy.sum(), leaf)
    within(grad, *want.grad([], torch.ones(5, device="cuda")), "entropy alone")


# --------------------------------------------------------------------- running
def test_another_stream_and_both_at_once(rs):
    x, g = rows_of(300, 20000, torch.bfloat16, 18)
    y, _ = rows_of(2, 200000, torch.bfloat16, 19)
    tx, ty = tokens_of(x, 1, g), tokens_of(y, 1, g)
    want = rs.token_logprobs(x, tx, 20), rs.token_logprobs(y, ty, 64)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        got = rs.token_logprobs(x, tx, 20, stream=a), rs.token_logprobs(y, ty, 64, stream=b)
        a.synchronize(), b.synchronize()
        for u, v in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(u, v))


def test_graph_replays_on_new_scores(rs):
    x, g = rows_of(40, 32000, torch.bfloat16, 20)
    t = tokens_of(x, 1, g)
    up = torch.ones(40, 1, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        rs.token_logprobs(x, t, 20)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = rs.token_logprobs(x, t, 20)
        grad = rs.token_logprobs_backward(x, got.stats, got.entropy, t, got.top_ids, up,
                                          temperature=1.0)
    for seed in (21, 22):
        x.copy_(rows_of(40, 32000, torch.bfloat16, seed)[0])
        graph.replay()
        torch.cuda.synchronize()
        want = rs.token_logprobs(x, t, 20)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.equal(grad, rs.token_logprobs_backward(x, want.stats, want.entropy, t,
                                                            want.top_ids, up))


def test_offsets_beyond_32_bits(rs):
    rows, cols = 33000, 131072  # 4.3e9 scores
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    for part in x.split(3000):
        part.normal_()
    t = torch.randint(0, cols, (rows,), device="cuda")
    got = rs.token_logprobs(x, t, 5)
    grad = rs.token_logprobs_backward(x, got.stats, got.entropy, t, grad_logprobs=torch.ones(rows, device="cuda"),
                                      grad_entropy=torch.ones(rows, device="cuda"))
    for r in (0, 16384, 32767, 32768, rows - 2):
        rest = x[r:r + 2]
        want = vo.Logprobs(rest, 1.0)
        within(got.entropy[r:r + 2], want.entropy, want.entropy_error, "entropy")
        assert torch.equal(got.top_ids[r:r + 2], want.top(5))
        logp, bound = want.logprobs(t[r:r + 2, None])
        within(got.logprobs[r:r + 2, None], logp, bound, "logprobs")
        ones = torch.ones(2, 1, device="cuda")
        g, bound = want.grad([(t[r:r + 2, None], ones)], ones[:, 0], None)
        within(grad[r:r + 2], g, bound, "gradient")


@pytest.mark.parametrize("top", [3, 200])
def test_one_row_of_many_scores(rs, top):
    x, g = rows_of(1, 100_000_003, torch.bfloat16, 22)
    check(rs, x, tokens_of(x, 2, g), top)


def test_same_bits_in_every_run(rs):
    x, g = rows_of(64, 131072, torch.bfloat16, 23)
    x[:, ::7] = 1.0
    t = tokens_of(x, 1, g)
    want = rs.token_logprobs(x, t, 100)
    for _ in range(10):
        assert all(torch.equal(a, b) for a, b in zip(rs.token_logprobs(x, t, 100), want))


def test_lists_teach_and_logprobs_weigh(rs):
    """What the calls return goes to the losses as it lies: a teacher's list is
    the same as one cut from sorted rows, and a policy's ratio to itself is 1."""
    x, g = rows_of(50, 4000, torch.bfloat16, 24)
    student, _ = rows_of(50, 4000, torch.bfloat16, 25)
    values, columns = rs.segmented_sort(x, descending=True)
    made = rs.token_logprobs(x, top=32)
    assert torch.equal(made.top_ids, columns[:, :32])
    a, _ = rs.distill_loss(student, values[:, :32], columns[:, :32], 2.0)
    b, _ = rs.distill_loss(student, made.top_logprobs, made.top_ids, 2.0)
    # the list's values differ by a constant of the row, and its rounding
    assert (a - b).abs().max() <= 4 * 64 * 2.0 ** -24 * made.top_logprobs.abs().max()
    t = tokens_of(x, 1, g)[:, 0].contiguous()
    old = rs.token_logprobs(x, t).logprobs
    adv = torch.randn(50, generator=g, device="cuda")
    losses, logp, _ = rs.policy_loss(x, t, old, adv)
    want = vo.Logprobs(x)
    error = 2 * want.logprobs(t[:, None])[1][:, 0]
    within(losses, -adv.double(), adv.double().abs() * 2 * error, "policy loss")
