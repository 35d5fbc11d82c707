"""The losses over the whole range of finite scores and temperatures: masks of
-1e10, -1e30 and the type's lowest value, in part of a row and in all of it,
large positive scores, small temperatures; every path of the row losses."""

import pytest
import torch

from tests import loss_bounds as lb

pytestmark = pytest.mark.gpu

# registers of one CTA (short, odd, 32 to 64 KB), and rows beyond: clusters,
# one CTA per row, few very long rows
SHAPES = [(16, 3000), (16, 2051), (304, 12000), (304, 30000), (16, 40000), (160, 40000), (8, 400003)]
FILLED = [(torch.bfloat16, (-1e10, -1e30, torch.finfo(torch.bfloat16).min)),
          (torch.float32, (-1e10, -1e30, torch.finfo(torch.float32).min))]


def scores(rows, cols, dtype, seed=0, spread=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(rows, cols, generator=g, device="cuda") * spread).to(dtype), g


def masked(x, fill):
    """Eight patterns of a finite mask, row after row; columns that stay."""
    cols = x.shape[1]
    kept = torch.ones_like(x, dtype=torch.bool)
    kept[0::8, :cols // 2] = False
    kept[1::8] = False                # the whole row
    kept[2::8, :1024] = False         # the first vectors of every thread, or of many
    kept[3::8, cols - 1024:] = False
    kept[4::8] = False
    kept[4::8, cols // 3] = True      # all but one
    kept[5::8, ::2] = False
    kept[6::8, 8:16] = False          # one vector
    return torch.where(kept, x, torch.full_like(x, fill)), kept


def some_columns(kept, k, g):
    """k columns that the mask leaves (any, where it leaves none); entries that
    would name a masked one are dropped."""
    draw = torch.rand(kept.shape, generator=g, device="cuda") + kept
    indices = draw.topk(k, dim=1).indices
    alive = kept.gather(1, indices) | ~kept.any(1, keepdim=True)
    return torch.where(alive, indices, torch.full_like(indices, -1))


def check_distill(rs, x, tau, indices, g, backward=False, grad_out=None, weights=None, rows=None):
    rows = lb.Rows(x, tau) if rows is None else rows
    values = torch.randn(indices.shape, generator=g, device="cuda") * min(tau, 1.0)
    losses, loss_bound, grad, bound, saved = lb.distill(rows, x, values, indices, weights)
    kw = {"temperature": tau, "weights": weights}
    lse_bound = rows.lse_error()
    fl, fs = rs.distill_loss(x, values, indices, **kw)
    if backward:
        got = rs.distill_loss_backward(None, x, fs, values, indices, **kw)
        lb.within(got, grad, bound + saved, "backward")
        over = x.clone()
        assert torch.equal(rs.distill_loss_backward(None, over, fs, values, indices, grad_out=over, **kw), got)
    gl, gs, gg = rs.distill_loss_grad(x, values, indices, grad_out=grad_out, **kw)
    lb.within(fl, losses, loss_bound, "losses")
    lb.within(gl, losses, loss_bound, "losses with gradient")
    on = torch.ones_like(rows.lse) if weights is None else (weights != 0).double()
    lb.within(fs, (rows.lse * on).float(), lse_bound, "lse")
    lb.within(gs, (rows.lse * on).float(), lse_bound, "lse with gradient")
    lb.within(gg, grad, bound, "gradient")


def check_policy(rs, x, tau, actions, g, backward=False, weights=None, rows=None,
                 kl=0.1):
    rows = lb.Rows(x, tau) if rows is None else rows
    n = x.shape[0]
    logp = -rows.dist.gather(1, actions.long()[:, None])[:, 0] - rows.log_sum
    old = (logp + torch.tensor([0.0, 0.1, -0.1, 0.5, -0.5], device="cuda").repeat(n)[:n]).float()
    ref = (logp + 0.3 * torch.randn(n, generator=g, device="cuda")).float()
    adv = torch.randn(n, generator=g, device="cuda")
    losses, loss_bound, logp, logp_bound, grad, bound, saved = lb.policy(rows, x, actions, old, adv, ref, kl=kl,
                                                                        weights=weights)
    kw = {"ref_logprobs": ref, "clip_low": 0.2, "clip_high": 0.28, "kl_coef": kl, "temperature": tau,
          "weights": weights}
    fl, fp, fs = rs.policy_loss(x, actions, old, adv, **kw)
    if backward:
        got = rs.policy_loss_backward(None, x, fs, actions, old, adv, **kw)
        lb.within(got, grad, bound + saved, "backward")
        over = x.clone()
        assert torch.equal(rs.policy_loss_backward(None, over, fs, actions, old, adv, grad_out=over, **kw), got)
    gl, gp, gs, gg = rs.policy_loss_grad(x, actions, old, adv, **kw)
    lb.within(fl, losses, loss_bound, "losses")
    lb.within(gl, losses, loss_bound, "losses with gradient")
    lb.within(fp, logp, logp_bound, "log-probabilities")
    lb.within(gp, logp, logp_bound, "log-probabilities with gradient")
    lb.within(fs, rows.lse.float(), rows.lse_error(), "lse")
    lb.within(gs, rows.lse.float(), rows.lse_error(), "lse with gradient")
    lb.within(gg, grad, bound, "gradient")


@pytest.mark.parametrize("dtype,fills", FILLED)
@pytest.mark.parametrize("tau", [0.7, 1.0, 2.0, 4.0])
@pytest.mark.parametrize("n,cols", SHAPES)
def test_finite_masks(rs, n, cols, tau, dtype, fills):
    for fill in fills:
        x, g = scores(n, cols, dtype, cols)
        x, kept = masked(x, fill)
        indices = some_columns(kept, 4, g)
        check_distill(rs, x, tau, indices, g)
        check_policy(rs, x, tau, indices.amax(1), g)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,cols", [(16, 3000), (304, 12000), (16, 40000), (160, 40000)])
def test_large_scores(rs, n, cols, dtype):
    """Rows of one large value, and rows with one above the others."""
    for size in (1e7, 1e9, 1e10, 1e20, 1e30):
        x, g = scores(n, cols, dtype, 1)
        x[0::3] = size
        x[1::3] = -size
        x[2::3, cols // 2] = size
        indices = torch.randint(0, cols, (n, 4), generator=g, device="cuda")
        indices[2::3] = cols // 2
        indices[2::3, 1:] = -1
        for tau in (0.5, 1.0, 3.0):
            check_distill(rs, x, tau, indices, g)
            check_policy(rs, x, tau, indices[:, 0].contiguous(), g)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("n,cols", [(16, 3000), (304, 12000), (16, 40000), (160, 40000)])
def test_small_temperatures(rs, n, cols, dtype):
    """Ordinary scores where only the largest counts."""
    for tau in (1e-3, 1e-6, 1e-9, 1e-15, 6e-20):
        x, g = scores(n, cols, dtype, 2)
        rows = lb.Rows(x, tau)
        indices = rows.q.topk(2, dim=1).indices
        indices[:, 1] = -1
        # gradients of the order of 1, which every type holds
        check_distill(rs, x, tau, indices, g, rows=rows, weights=torch.full((n,), 1 / tau, device="cuda"))
        check_policy(rs, x, tau, indices[:, 0].contiguous(), g, rows=rows,
                     weights=torch.full((n,), tau, device="cuda"))


def balance64(x, ids, mask=None):
    """(loss, mean probabilities, gradient, scale of its terms) in 64 bits."""
    n, experts = x.shape
    kept = torch.ones(n, dtype=torch.bool, device="cuda") if mask is None else mask
    z = x.double()
    p = (z - z.amax(1, keepdim=True)).exp()
    p = p / p.sum(1, keepdim=True) * kept[:, None]
    tokens = max(int(kept.sum()), 1)
    counts = torch.bincount(ids[kept].reshape(-1), minlength=experts).double()
    share = counts * experts / (ids.shape[1] * tokens)
    mean = p.sum(0) / tokens
    dot = (p @ share)[:, None]
    return share @ mean, mean, p * (share - dot) / tokens, p * (share + dot) / tokens


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("tokens,experts", [(40, 20), (37, 8), (300, 64), (5000, 60), (6000, 128), (999, 257)])
def test_balance_of_large_finite_scores(rs, tokens, experts, dtype):
    """Tokens of equal scores are spread evenly, masked experts get nothing, and
    no token drops out, however large the finite scores are."""
    lowest = torch.finfo(dtype).min
    for size in (-1e9, -1e10, -1e15, -1e20, -1e30, 1e10, 1e30, lowest, -lowest, -40000.0):
        if abs(size) > -lowest:
            continue
        x, g = scores(tokens, experts, dtype, experts, 2.0)
        x[0::5] = size                       # equal scores
        x[1::5, experts // 2:] = min(size, -size)
        x[2::5, 1:] = min(size, -size)
        x[3::5, experts // 3] = max(size, -size)
        ids = torch.randint(0, experts, (tokens, 2), generator=g, device="cuda")
        mask = torch.rand(tokens, generator=g, device="cuda") < 0.8
        for kept in (None, mask):
            loss, mean, grad, terms = balance64(x, ids, kept)
            out = rs.balance_loss_grad(x, ids, token_mask=kept)
            back = rs.balance_loss_backward(None, x, out[1], out[3], 2, token_mask=kept)
            only = rs.balance_loss(x, ids, token_mask=kept)
            # a probability: its exponent's rounding over a spread of 16 nats,
            # or over the 2^6 by which a large origin's product may be off;
            # sums of up to 32 per lane and 5 steps; then sums over tokens
            u = 2.0 ** -24 * (2 * 64 + 64 + 40)
            for got in (out, only):
                lb.within(got[2], mean, mean * (u + 2.0 ** -24 * (tokens / 8 + 64)) + 2.0 ** -60, "mean_probs")
                lb.within(got[0], loss, loss * (u + 2.0 ** -24 * (tokens / 8 + experts + 64)), "loss")
            round_to, tiny = {torch.bfloat16: (2.0 ** -8, 0), torch.float16: (2.0 ** -11, 2.0 ** -24),
                              torch.float32: (2.0 ** -24, 0)}[dtype]
            bound = terms * (2 * u + 32 * 2.0 ** -24) + grad.abs() * round_to * 1.01 + tiny + 2.0 ** -60
            lb.within(out[4], grad, bound, "gradient")
            lb.within(back, grad, bound, "backward")


@pytest.mark.parametrize("dtype,fills", FILLED)
@pytest.mark.parametrize("n,cols", [(16, 3000), (304, 12000), (16, 40000), (160, 40000)])
def test_targets_on_masked_columns(rs, n, cols, dtype, fills):
    """A teacher's entry on a column that the student masks: its loss is as
    large as the mask, and infinite only where a float cannot hold it."""
    for fill in fills:
        x, g = scores(n, cols, dtype, 5)
        x, kept = masked(x, fill)
        indices = torch.rand(n, cols, generator=g, device="cuda").topk(4, dim=1).indices
        indices[0::8, 0] = 3          # masked
        indices[0::8, 1:] = -1        # nothing but it
        for tau in (0.1, 0.25, 0.7, 1.0, 3.0, 1e20):
            rows = lb.Rows(x, tau)
            weights = torch.full((n,), 0.125 / min(tau, 1e19), device="cuda")
            values = torch.randn(n, 4, generator=g, device="cuda")
            want, bound, _, _, _ = lb.distill(rows, x, values, indices, weights)
            kw = {"temperature": tau, "weights": weights}
            for got in (rs.distill_loss(x, values, indices, **kw)[0],
                        rs.distill_loss_grad(x, values, indices, **kw)[0]):
                lb.within(got, want.float(), bound, f"losses at {fill}, {tau}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,cols", SHAPES + [(1, 200000)])
def test_backward_of_rows_whose_lse_says_too_little(rs, n, cols, dtype):
    """A saved lse of -1e10 has lost the logarithm of the sum, one of the type's
    lowest value over a temperature below 1 is -inf: the gradient is right all
    the same, also over the logits."""
    lowest = torch.finfo(dtype).min
    for fill, tau in ((-1e10, 1.0), (-1e30, 2.0), (lowest, 0.7), (lowest, 1.0), (lowest, 4.0), (-3000.0, 1.0),
                      (-300.0, 0.25)):
        x, g = scores(n, cols, dtype, cols)
        x, kept = masked(x, fill)
        indices = some_columns(kept, 4, g)
        check_distill(rs, x, tau, indices, g, backward=True)
        check_policy(rs, x, tau, indices.amax(1), g, backward=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("n,cols", [(16, 3000), (304, 12000), (16, 40000), (160, 40000), (2, 300007)])
def test_backward_at_small_temperatures(rs, n, cols, dtype):
    for tau in (1e-3, 1e-6, 1e-15, 6e-20):
        x, g = scores(n, cols, dtype, 2)
        x[1::4, ::5] = torch.finfo(dtype).min
        rows = lb.Rows(x, tau)
        indices = rows.q.topk(2, dim=1).indices
        indices[:, 1] = -1
        check_distill(rs, x, tau, indices, g, True, rows=rows, weights=torch.full((n,), 1 / tau, device="cuda"))
        check_policy(rs, x, tau, indices[:, 0].contiguous(), g, True, rows=rows,
                     weights=torch.full((n,), tau, device="cuda"))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,cols", [(64, 65536), (200, 65536), (64, 3000), (12, 400000)])
def test_losses_near_zero(rs, n, cols, dtype):
    """One score far above the others and far behind the first, which the
    target names: the loss is some 1e-5, and off by the rounding of numbers
    near 1 (16 units: two exponentials of 2 ulp, sums, a logarithm), however far
    the scores before it lie below."""
    x, g = scores(n, cols, dtype, 7, 1.0)
    at = torch.randint(cols * 3 // 4, cols, (n, 1), generator=g, device="cuda")
    height = 10.4 + torch.logsumexp(x.double(), 1, keepdim=True)
    x.scatter_(1, at, (height + torch.rand(n, 1, generator=g, device="cuda")).to(dtype))
    want = torch.logsumexp(x.double(), 1) - x.double().gather(1, at)[:, 0]
    assert 5e-6 < float(want.min()) and float(want.max()) < 1e-4
    bound = torch.full_like(want, 16 * 2.0 ** -24)
    values = torch.zeros(n, 1, device="cuda")
    zeros = torch.zeros(n, device="cuda")
    for got in (rs.distill_loss(x, values, at)[0], rs.distill_loss_grad(x, values, at)[0],
                -rs.policy_loss(x, at[:, 0], zeros, zeros)[1],
                -rs.policy_loss_grad(x, at[:, 0], zeros, zeros)[1]):
        lb.within(got, want, bound, "losses")
