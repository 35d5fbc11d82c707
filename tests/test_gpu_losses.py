"""The losses over rows of scores against their formulas in 64 bits: types,
odd and long rows, strides and alignments, masks, dropped and repeated
entries, -inf and NaN, other streams, graphs, and the gradient against
differences of the loss itself."""
import math

import pytest
import torch

from tests import loss_oracle as lo

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]


def rows_of(rows, cols, dtype, seed, pad=0, shift=0, spread=3.0):
    """(cpu scores, the same on the GPU as a view with padded rows that starts
    `shift` elements into its buffer; the padding holds NaN)."""
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, cols, generator=g) * spread).to(dtype)
    buf = torch.full((rows * (cols + pad) + shift,), math.nan, dtype=dtype, device="cuda")
    view = buf[shift:].as_strided((rows, cols), (cols + pad, 1), shift)
    view.copy_(x.cuda())
    return x, view, g


def distill_case(x, k, g, short=True):
    rows, cols = x.shape
    values, indices = torch.topk(x.float() + torch.randn(x.shape, generator=g), k, dim=1)
    if short and k > 1:  # some rows' lists end earlier
        length = torch.randint(1, k + 1, (rows, 1), generator=g)
        indices = torch.where(torch.arange(k) < length, indices, torch.full_like(indices, -1))
    return values.to(x.dtype), indices


def check_distill(rs, x, xd, values, indices, tau=1.0, weights=None, up=None, grad_out=None):
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    losses, lse, grad, size = lo.distill(x, values, indices, tau, weights)
    err = lo.row_error(x, tau)
    ones = torch.ones(x.shape[0], dtype=torch.float64)
    w = (ones if weights is None else weights.double()).abs() * tau * tau
    loss_bound = w * (2 * err + 2 * lo.row_error(values.float(), tau)) + 16 * lo.U32 * losses.abs()
    args = (dev(values), dev(indices))
    kw = {"temperature": tau, "weights": dev(weights)}
    fl, fs = rs.distill_loss(xd, *args, **kw)
    bound = lo.grad_bound(grad, size, err + lo.row_error(values.float(), tau), x.dtype)
    # the backward call first: a gradient may be asked to lie over the logits
    gb = rs.distill_loss_backward(None, xd, fs, *args, **kw)
    lo.assert_within(gb, grad, bound, "backward")
    if up is not None:
        _, _, grad_up, size_up = lo.distill(x, values, indices, tau, weights, up)
        gu = rs.distill_loss_backward(dev(up), xd, fs, *args, **kw)
        lo.assert_within(gu, grad_up, lo.grad_bound(
            grad_up, size_up, err + lo.row_error(values.float(), tau), x.dtype), "upstream")
    gl, gs, gg = rs.distill_loss_grad(xd, *args, grad_out=grad_out, **kw)
    for got, want, b, what in ((fl, losses, loss_bound, "losses"), (fs, lse, err, "lse"),
                               (gl, losses, loss_bound, "losses with grad"),
                               (gs, lse, err, "lse with grad"), (gg, grad, bound, "grad")):
        lo.assert_within(got, want, b, what)
    return gg


def check_policy(rs, x, xd, actions, old, adv, ref=None, kl=0.0, low=0.2, high=0.28, tau=1.0,
                 weights=None, up=None):
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    losses, logp, lse, grad, size, loss_size = lo.policy(x, actions, old, adv, ref, low, high, kl,
                                                         tau, weights)
    err = lo.row_error(x, tau)
    args = (dev(actions), dev(old), dev(adv))
    kw = {"ref_logprobs": dev(ref), "clip_low": low, "clip_high": high, "kl_coef": kl,
          "temperature": tau, "weights": dev(weights)}
    loss_bound = loss_size * (err + 16 * lo.U32)
    bound = lo.grad_bound(grad, size, 2 * err, x.dtype)
    fl, fp, fs = rs.policy_loss(xd, *args, **kw)
    gb = rs.policy_loss_backward(None, xd, fs, *args, **kw)
    lo.assert_within(gb, grad, bound, "backward")
    if up is not None:
        _, _, _, grad_up, size_up, _ = lo.policy(x, actions, old, adv, ref, low, high, kl, tau,
                                                 weights, up)
        gu = rs.policy_loss_backward(dev(up), xd, fs, *args, **kw)
        lo.assert_within(gu, grad_up, lo.grad_bound(grad_up, size_up, 2 * err, x.dtype), "upstream")
    gl, gp, gs, gg = rs.policy_loss_grad(xd, *args, **kw)
    for got, want, b, what in ((fl, losses, loss_bound, "losses"), (fp, logp, err, "logprobs"),
                               (fs, lse, err, "lse"), (gl, losses, loss_bound, "losses with grad"),
                               (gp, logp, err, "logprobs with grad"), (gs, lse, err, "lse with grad"),
                               (gg, grad, bound, "grad")):
        lo.assert_within(got, want, b, what)


def check_balance(rs, x, xd, ids, mask=None, scale=1.0):
    loss, counts, mean, n, grad, size = lo.balance(x, ids, mask, scale)
    dev = None if mask is None else mask.cuda()
    live = x[mask.bool()] if mask is not None else x
    err = float(lo.row_error(live, 1.0).max()) if live.shape[0] else 0.0
    # sums over tokens: each lane adds one token after another, at most tokens
    # of them, then per-warp and per-CTA sums
    total = err + lo.U32 * (x.shape[0] + 1024)
    f = rs.balance_loss(xd, ids.cuda(), token_mask=dev)
    g = rs.balance_loss_grad(xd, ids.cuda(), token_mask=dev, scale=scale)
    for out in (f, g):
        assert out[1].cpu().tolist() == counts.tolist()
        assert out[3].cpu().tolist() == [n]
        lo.assert_within(out[2], mean, mean.abs() * total, "mean_probs")
        lo.assert_within(out[0], torch.tensor(loss, dtype=torch.float64), abs(loss) * (total + 64 * lo.U32),
                         "loss")
    bound = lo.grad_bound(grad, size, torch.full((x.shape[0],), 2 * err + 1024 * lo.U32), x.dtype)
    lo.assert_within(g[4], grad, bound, "grad")
    up = torch.full((1,), scale, device="cuda")
    gb = rs.balance_loss_backward(up, xd, f[1], f[3], ids.shape[1], token_mask=dev)
    lo.assert_within(gb, grad, bound, "backward")


def policy_inputs(x, tau, g):
    rows, cols = x.shape
    actions = torch.randint(0, cols, (rows,), generator=g)
    logp = torch.log_softmax(x.double() / tau, 1).gather(1, actions[:, None])[:, 0]
    old = (logp + torch.tensor([0.0, 0.1, -0.1, 0.5, -0.5]).repeat(rows)[:rows]).float()
    ref = (logp + 0.3 * torch.randn(rows, generator=g)).float()
    return actions, old, ref, torch.randn(rows, generator=g)


# widths around vectors, warps, tiles and cluster limits
WIDTHS = [(1, 1), (3, 2), (2, 7), (5, 8), (3, 31), (4, 33), (3, 255), (2, 1000), (3, 4097),
          (2, 8191), (2, 16384), (2, 50001), (1, 65536), (2, 131075), (1, 300007)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", WIDTHS)
def test_distill_widths(rs, rows, cols, dtype):
    x, xd, g = rows_of(rows, cols, dtype, rows + cols)
    values, indices = distill_case(x, min(cols, 9), g)
    check_distill(rs, x, xd, values, indices)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", WIDTHS)
def test_policy_widths(rs, rows, cols, dtype):
    x, xd, g = rows_of(rows, cols, dtype, rows + cols)
    actions, old, ref, adv = policy_inputs(x, 1.0, g)
    check_policy(rs, x, xd, actions, old, adv, ref, 0.05)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,shift", [(1, 0), (0, 1), (3, 5), (64, 8), (7, 7)])
def test_strides_and_alignments(rs, dtype, pad, shift):
    for cols in (1003, 20001):
        x, xd, g = rows_of(5, cols, dtype, pad + shift, pad, shift)
        values, indices = distill_case(x, 5, g)
        check_distill(rs, x, xd, values, indices)
        # a gradient whose rows are aligned otherwise than the logits'
        buf = torch.full((5 * (cols + 9) + 3,), 7.0, dtype=dtype, device="cuda")
        out = buf[3:].as_strided((5, cols), (cols + 9, 1), 3)
        check_distill(rs, x, xd, values, indices, grad_out=out)
        gaps = buf[3:3 + 5 * (cols + 9)].view(5, cols + 9)[:, cols:]
        assert bool((gaps == 7.0).all()) and bool((buf[:3] == 7.0).all())
        actions, old, ref, adv = policy_inputs(x, 1.0, g)
        check_policy(rs, x, xd, actions, old, adv, ref, 0.1)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(700, 515), (400, 9000), (161, 40000)])
def test_many_rows(rs, rows, cols, dtype):
    """More rows than the GPU holds at once, some masked."""
    x, xd, g = rows_of(rows, cols, dtype, 5)
    weights = torch.rand(rows, generator=g)
    weights[torch.randperm(rows, generator=g)[:rows // 4]] = 0.0
    values, indices = distill_case(x, 16, g)
    check_distill(rs, x, xd, values, indices, 1.0, weights)
    actions, old, ref, adv = policy_inputs(x, 1.0, g)
    check_policy(rs, x, xd, actions, old, adv, ref, 0.05, weights=weights)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tau", [0.25, 0.7, 3.0])
def test_temperature_weights_upstream(rs, dtype, tau):
    x, xd, g = rows_of(6, 3001, dtype, 11)
    weights = torch.tensor([1.0, 0.0, -0.5, 2.0, 0.0, 0.125])
    up = torch.tensor([1.0, 2.0, 0.5, 0.0, 1.0, -3.0])
    values, indices = distill_case(x, 7, g)
    check_distill(rs, x, xd, values, indices, tau, weights, up)
    actions, old, ref, adv = policy_inputs(x, tau, g)
    check_policy(rs, x, xd, actions, old, adv, ref, 0.05, tau=tau, weights=weights, up=up)
    check_policy(rs, x, xd, actions, old, adv, None, 0.0, tau=tau, weights=weights, up=up)


@pytest.mark.parametrize("k", [1, 2, 31, 32, 33, 64, 255, 1023, 1024])
def test_list_lengths(rs, k):
    x, xd, g = rows_of(3, 2048, torch.bfloat16, k)
    values, indices = distill_case(x, k, g)
    check_distill(rs, x, xd, values, indices)
    check_distill(rs, x, xd, values.float(), indices.int())  # other list types


def test_lists_of_a_descending_row_sort(rs):
    """The first k columns of what segmented_sort returns, as they lie there."""
    x, xd, g = rows_of(4, 9000, torch.bfloat16, 2)
    teacher = (x.float() + torch.randn(x.shape, generator=g)).to(torch.bfloat16)
    values, indices = rs.segmented_sort(teacher.cuda(), descending=True)
    got = rs.distill_loss_grad(xd, values[:, :20], indices[:, :20])
    losses, _, grad, size = lo.distill(x, values[:, :20].cpu(), indices[:, :20].cpu())
    err = lo.row_error(x, 1.0) + lo.row_error(values[:, :20].cpu(), 1.0)
    lo.assert_within(got[0], losses, 2 * err, "losses")
    lo.assert_within(got[2], grad, lo.grad_bound(grad, size, err, torch.bfloat16), "grad")


@pytest.mark.parametrize("k", [5, 100, 700])
def test_repeated_columns(rs, k):
    """A column named more than once gets the probability of each entry."""
    x, xd, g = rows_of(4, 1500, torch.float32, 3)
    values = torch.randn(4, k, generator=g)
    indices = torch.randint(0, 1500, (4, k), generator=g)
    indices[0] = 17                                   # one column only
    indices[1] = torch.arange(k) // 2                 # pairs
    indices[2, k // 2:] = indices[2, :k - k // 2].clone()  # far apart
    indices[3, ::3] = -1
    check_distill(rs, x, xd, values, indices)


def test_rows_without_targets(rs):
    x, xd, g = rows_of(6, 600, torch.float16, 4)
    values, indices = distill_case(x, 6, g, short=False)
    indices[0] = -1                       # nothing named
    indices[1] = 600                      # just outside
    indices[2, 1:] = 2 ** 40              # far outside, beyond 32 bits
    indices[3] = -2 ** 62
    values[4] = -math.inf                 # named, but of no probability
    values[5, 2] = -math.inf
    check_distill(rs, x, xd, values, indices)
    actions = torch.tensor([-1, 600, 2 ** 40, -100, 0, 599])
    z = torch.zeros(6)
    check_policy(rs, x, xd, actions, torch.log_softmax(x.double(), 1)[:, 0].float(), z + 1, z - 3, 0.1)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("cols", [40, 3000, 70000])
def test_masked_scores(rs, dtype, cols):
    """-inf and the type's lowest value, in part of a row, first, last, and
    in all of it."""
    low = torch.finfo(dtype).min
    x, xd, g = rows_of(9, cols, dtype, 8)
    x[0, :cols // 2] = -math.inf
    x[1, cols // 2:] = -math.inf
    x[2] = -math.inf
    x[3, 1:] = -math.inf
    x[4, :-1] = -math.inf
    x[5, ::2] = low
    x[6] = low
    x[7, 5:] = low
    x[8, ::3] = -math.inf
    xd.copy_(x.cuda())
    indices = torch.stack([torch.randperm(cols, generator=g)[:4] for _ in range(9)])
    indices[0, 0], indices[1, 0], indices[3], indices[4] = cols - 1, 0, 0, cols - 1
    values = torch.randn(9, 4, generator=g)
    check_distill(rs, x, xd, values, indices)
    actions = torch.tensor([cols - 1, 0, 3, 0, cols - 1, 1, 7, 2, 1])
    logp = torch.log_softmax(x.double(), 1).gather(1, actions[:, None])[:, 0]
    old = (logp + 0.05).nan_to_num().float()
    check_policy(rs, x, xd, actions, old, torch.ones(9), old, 0.1)


def test_action_of_no_probability(rs):
    x, xd, _ = rows_of(2, 100, torch.float32, 8)
    x[:, 5] = -math.inf
    xd.copy_(x.cuda())
    out = rs.policy_loss_grad(xd, torch.tensor([5, 5], device="cuda"), torch.zeros(2, device="cuda") - 5,
                              torch.tensor([1.0, -1.0], device="cuda"))
    assert out[0].tolist() == pytest.approx([0.0, 0.8]) and out[1].tolist() == [-math.inf] * 2
    assert bool((out[3] == 0).all())


@pytest.mark.parametrize("cols", [50, 5000, 70000])
@pytest.mark.parametrize("dtype", TYPES)
def test_nan_and_inf_stay_in_their_rows(rs, dtype, cols):
    x, xd, g = rows_of(6, cols, dtype, 9)
    x[1, cols // 3] = math.nan
    x[3, cols - 1] = math.inf
    x[4, 0] = math.nan  # of weight 0: not read
    xd.copy_(x.cuda())
    weights = torch.tensor([1.0, 1.0, 1.0, 1.0, 0.0, 1.0])
    values, indices = distill_case(x.nan_to_num(0, 0, 0), 4, g)
    bad = [1, 3]
    good = [0, 2, 4, 5]
    losses, lse, grad = rs.distill_loss_grad(xd, values.cuda(), indices.cuda(), weights=weights.cuda())
    assert losses[bad].isnan().all() and lse[bad].isnan().all() and grad[bad].isnan().all()
    want = lo.distill(x[good], values[good], indices[good], 1.0, weights[good])
    err = lo.row_error(x[good].nan_to_num(0), 1.0) + lo.row_error(values[good], 1.0)
    lo.assert_within(grad[good], want[2], lo.grad_bound(want[2], want[3], err, dtype), "grad")
    actions, old, ref, adv = policy_inputs(x.nan_to_num(0, 0, 0), 1.0, g)
    out = rs.policy_loss_grad(xd, actions.cuda(), old.cuda(), adv.cuda(), ref.cuda(), kl_coef=0.1,
                              weights=weights.cuda())
    for t in (out[0], out[1], out[2], out[3]):
        assert t[bad].isnan().all() and not t[good].isnan().any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("cols", [9, 2050, 40003])
def test_gradient_over_the_logits(rs, dtype, cols):
    x, xd, g = rows_of(5, cols, dtype, 10, pad=3, shift=1)
    values, indices = distill_case(x, 6, g)
    args = values.cuda(), indices.cuda()
    want = rs.distill_loss_grad(xd, *args)
    y = xd.as_strided(xd.shape, xd.stride(), xd.storage_offset())
    base = xd.clone()
    got = rs.distill_loss_grad(y, *args, grad_out=y)
    assert got[2].data_ptr() == xd.data_ptr()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    z = base.clone()
    lse = want[1]
    assert torch.equal(rs.distill_loss_backward(None, z, lse, *args, grad_out=z),
                       rs.distill_loss_backward(None, base, lse, *args))
    ids = torch.randint(0, cols, (5, 2), generator=g).cuda()
    if cols <= 1024:
        w = rs.balance_loss_grad(base, ids)
        z = base.clone()
        assert torch.equal(rs.balance_loss_grad(z, ids, grad_out=z)[4], w[4])


def test_same_bits_every_time(rs):
    x, xd, g = rows_of(300, 20011, torch.bfloat16, 12)
    values, indices = distill_case(x, 33, g)
    args = xd, values.cuda(), indices.cuda()
    first = rs.distill_loss_grad(*args)
    router = torch.randn(5000, 60, generator=g).cuda()
    ids = torch.topk(router, 4).indices
    bal = rs.balance_loss_grad(router, ids)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, rs.distill_loss_grad(*args)))
        assert all(torch.equal(a, b) for a, b in zip(bal, rs.balance_loss_grad(router, ids)))


def test_gradient_against_differences(rs):
    """Central differences of the kernel's own loss along random directions:
    the loss's error (row_error) over the step, and the step's square."""
    x, xd, g = rows_of(4, 700, torch.float32, 13, spread=1.0)
    values, indices = distill_case(x, 5, g)
    actions, old, ref, adv = policy_inputs(x, 1.0, g)
    d = torch.randn(4, 700, generator=g).cuda()
    h = 2.0 ** -7
    err = float(lo.row_error(x, 1.0).max())
    args = values.cuda(), indices.cuda()
    grad = rs.distill_loss_grad(xd, *args)[2]
    diff = (rs.distill_loss(xd + h * d, *args)[0] - rs.distill_loss(xd - h * d, *args)[0]) / (2 * h)
    # third derivatives along d are at most of the order of max|d|^3 < 64
    tol = 64 * h * h + 4 * err / h
    assert bool(((grad * d).sum(1) - diff).abs().max() < tol)
    kw = {"ref_logprobs": ref.cuda(), "kl_coef": 0.2, "clip_low": 0.9, "clip_high": 9.0}
    args = actions.cuda(), old.cuda(), adv.cuda()
    grad = rs.policy_loss_grad(xd, *args, **kw)[3]
    diff = (rs.policy_loss(xd + h * d, *args, **kw)[0]
            - rs.policy_loss(xd - h * d, *args, **kw)[0]) / (2 * h)
    assert bool(((grad * d).sum(1) - diff).abs().max() < 4 * tol)


def test_autograd(rs):
    x, xd, g = rows_of(5, 900, torch.float32, 14)
    values, indices = (t.cuda() for t in distill_case(x, 6, g))
    actions, old, ref, adv = (t.cuda() for t in policy_inputs(x, 1.0, g))
    leaf = xd.clone().requires_grad_(True)
    up = torch.rand(5, generator=g).cuda()
    losses, lse = rs.distill_loss(leaf, values, indices, 2.0)
    (losses * up).sum().backward()
    assert torch.equal(leaf.grad, rs.distill_loss_backward(up, xd, lse, values, indices, 2.0))
    leaf.grad = None
    losses, logprobs, lse = rs.policy_loss(leaf, actions, old, adv, ref, kl_coef=0.1)
    assert not logprobs.requires_grad
    losses.mean().backward()
    want = rs.policy_loss_backward(torch.full((5,), 0.2, device="cuda"), xd, lse, actions, old, adv,
                                   ref, kl_coef=0.1)
    assert torch.equal(leaf.grad, want)
    router = torch.randn(50, 12, generator=g).cuda().requires_grad_(True)
    ids = torch.topk(router.detach(), 3).indices
    loss, counts, mean, n = rs.balance_loss(router, ids)
    (loss * 0.01).backward()
    want = rs.balance_loss_backward(torch.tensor([0.01], device="cuda"), router.detach(), counts, n, 3)
    assert torch.equal(router.grad, want)
    with pytest.raises(ValueError, match="outputs or a stream"):
        rs.distill_loss(leaf, values, indices, losses_out=torch.empty(5, device="cuda"))


def test_other_stream(rs):
    x, xd, g = rows_of(64, 30000, torch.bfloat16, 15)
    values, indices = (t.cuda() for t in distill_case(x, 8, g))
    want = rs.distill_loss_grad(xd, values, indices)
    router = torch.randn(3000, 33, generator=g).cuda()
    ids = torch.topk(router, 2).indices
    bal = rs.balance_loss_grad(router, ids)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        got = rs.distill_loss_grad(xd, values, indices, stream=s)
        gb = rs.balance_loss_grad(router, ids, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(a, b) for a, b in zip(gb, bal))


def test_cuda_graph(rs):
    x, xd, g = rows_of(40, 12001, torch.float16, 16)
    values, indices = (t.cuda() for t in distill_case(x, 8, g))
    router = torch.randn(2000, 24, generator=g).cuda()
    ids = torch.topk(router, 2).indices
    rs.distill_loss_grad(xd, values, indices)
    rs.balance_loss_grad(router, ids)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = rs.distill_loss_grad(xd, values, indices)
        gb = rs.balance_loss_grad(router, ids)
    for seed in (1, 2):
        xd.copy_(torch.randn(40, 12001, generator=torch.Generator().manual_seed(seed)).cuda())
        router.mul_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, rs.distill_loss_grad(xd, values, indices)))
        assert all(torch.equal(a, b) for a, b in zip(gb, rs.balance_loss_grad(router, ids)))


def test_graph_of_long_rows(rs):
    """Rows taken over from unlaunched CTAs, replayed: more rows than SMs."""
    x, xd, g = rows_of(400, 33000, torch.bfloat16, 17)
    actions, old, ref, adv = (t.cuda() for t in policy_inputs(x, 1.0, g))
    rs.policy_loss_grad(xd, actions, old, adv, ref, kl_coef=0.1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = rs.policy_loss_grad(xd, actions, old, adv, ref, kl_coef=0.1)
    for _ in range(3):
        xd.mul_(0.75)
        graph.replay()
        torch.cuda.synchronize()
        want = rs.policy_loss_grad(xd, actions, old, adv, ref, kl_coef=0.1)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("rows,cols", [(1, 90000), (5, 90000), (200, 90000), (3, 400000), (160, 400000)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_beyond_the_ring(rs, rows, cols, dtype):
    """Rows that one CTA cannot hold, alone and as many as there are SMs,
    against the gradient of plain double arithmetic."""
    g = torch.Generator(device="cuda").manual_seed(rows + cols)
    x = (torch.randn(rows, cols, generator=g, device="cuda") * 3).to(dtype)
    values, indices = torch.topk(x.float() + torch.randn(x.shape, generator=g, device="cuda"), 40, dim=1)
    weights = torch.rand(rows, generator=g, device="cuda")
    weights[::7] = 0
    losses, lse, grad = rs.distill_loss_grad(x, values, indices, weights=weights)
    back = rs.distill_loss_backward(None, x, lse, values, indices, weights=weights)
    err = lo.row_error(torch.tensor([[-16.0, 16.0]]).expand(1, 2), 1.0)[0] + lo.U32 * cols / 32
    u, tiny = lo.ROUND[dtype]
    for r in range(rows):
        z = x[r].double()
        logq = z - torch.logsumexp(z, 0)
        logp = torch.log_softmax(values[r].double(), 0)
        w = weights[r].double()
        target = torch.zeros_like(z).index_add_(0, indices[r], logp.exp())
        want = w * (logq.exp() - target)
        bound = w * (logq.exp() + target) * (2 * float(err) + 16 * lo.U32) + want.abs() * u * 1.01 + tiny
        for got in (grad[r], back[r]):
            assert bool(((got.double() - want).abs() <= bound).all()), (r, "gradient")
        loss = w * (logp.exp() * (logp - logq[indices[r]])).sum()
        assert abs(losses[r].double() - loss) <= 4 * float(err) * (1 + abs(loss)), (r, "loss")


@pytest.mark.parametrize("k", [300, 1024])
def test_long_lists_of_long_rows(rs, k):
    """Long lists leave less of the ring; some columns are named twice."""
    x, xd, g = rows_of(6, 70001, torch.bfloat16, k)
    values, indices = distill_case(x, k, g)
    indices[1, 1::2] = indices[1, 0::2]
    indices[4, k // 2] = indices[4, 0]
    check_distill(rs, x, xd, values, indices)


@pytest.mark.parametrize("rows,cols,dtype", [(1000, 65536, torch.bfloat16), (1000, 100003, torch.float16),
                                             (160, 400000, torch.float32)])
def test_long_rows_give_the_same_bits_under_load(rs, rows, cols, dtype):
    """Copies run ahead of the threads that read the slots: a slot that is given
    back too early would show as a line of another row's gradient, now and then
    and only while memory is busy."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = (torch.randn(rows, cols, generator=g, device="cuda") * 3).to(dtype)
    values, indices = torch.topk(x, 40, dim=1)
    first = rs.distill_loss_grad(x, values, indices)
    for _ in range(40):
        again = rs.distill_loss_grad(x, values, indices)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_a_wait_that_runs_out_is_reported(rs):
    assert rs.row_wait_timeout_probe(3_000_000) == rs.RS_ERR_LOOKBACK_TIMEOUT
    x, xd, g = rows_of(3, 40000, torch.bfloat16, 18)  # and the next call is right
    values, indices = distill_case(x, 4, g)
    check_distill(rs, x, xd, values, indices)


def test_int32_actions_and_indices(rs):
    x, xd, g = rows_of(5, 4000, torch.float16, 19)
    actions, old, ref, adv = policy_inputs(x, 1.0, g)
    actions[2] = -1
    check_policy(rs, x, xd, actions.int(), old, adv, ref, 0.1)


def test_the_example_trains(rs):
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "train_step.py")
    spec = importlib.util.spec_from_file_location("train_step", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    history = example.main(steps=12)
    assert history["distill"][-1] < 0.8 * history["distill"][0]
    assert 0.9 < history["balance"][-1] < 3.0
    assert history["reward"][-1] >= history["reward"][0] - 0.05
    assert all(math.isfinite(v) for series in history.values() for v in series)


# --------------------------------------------------------------- balance
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,experts,k", [
    (1, 1, 1), (1, 8, 2), (7, 3, 1), (33, 8, 2), (100, 16, 4), (65, 17, 3), (1000, 60, 4),
    (513, 64, 8), (257, 100, 6), (300, 128, 1), (777, 160, 6), (4100, 256, 8), (90, 257, 5),
    (50, 384, 8), (40, 512, 8), (37, 1000, 3), (21, 1024, 16), (20000, 8, 2)])
def test_balance_shapes(rs, tokens, experts, k, dtype):
    x, xd, g = rows_of(tokens, experts, dtype, tokens)
    ids = torch.topk(x.float(), min(k, experts), dim=1).indices
    check_balance(rs, x, xd, ids, scale=0.01 * tokens)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("experts,pad,shift", [(8, 1, 0), (64, 3, 1), (64, 8, 8), (100, 0, 2), (256, 5, 5)])
def test_balance_strides_masks_and_drops(rs, dtype, experts, pad, shift):
    x, xd, g = rows_of(331, experts, dtype, experts, pad, shift)
    order = torch.argsort(x.float(), dim=1, descending=True)
    mask = torch.rand(331, generator=g) < 0.7
    for ids in (order[:, :3], order[:, :3].contiguous().int()):  # as a sort leaves them; packed
        check_balance(rs, x, xd, ids, mask, 3.0)
    ids = order[:, :4].clone()
    ids[::3, 1] = -1
    ids[1::3, 2] = experts
    ids[2::5] = 2 ** 40
    ids[4::7, 3] = ids[4::7, 0]  # named twice
    x2 = x.clone()
    x2[~mask] = math.nan  # padded tokens are not read
    xd.copy_(x2.cuda())
    check_balance(rs, x, xd, ids, mask, 3.0)
    check_balance(rs, x, xd, ids, mask.to(torch.uint8), -0.5)


def test_balance_masked_scores_and_empty(rs):
    x, xd, g = rows_of(40, 20, torch.float32, 6)
    x[3] = -math.inf
    x[4, 1:] = -math.inf
    x[5, ::2] = torch.finfo(torch.float32).min
    x[6] = torch.finfo(torch.float32).min
    xd.copy_(x.cuda())
    ids = torch.topk(torch.randn(40, 20, generator=g), 2).indices
    check_balance(rs, x, xd, ids)
    check_balance(rs, x, xd, ids, torch.zeros(40, dtype=torch.bool))  # nothing kept
    out = rs.balance_loss(xd[:0], ids[:0].cuda())
    assert out[0].item() == 0 and not out[1].any() and not out[2].any() and out[3].item() == 0
    out = rs.balance_loss_grad(xd[:0], ids[:0].cuda())
    assert out[4].shape == (0, 20) and out[0].item() == 0


@pytest.mark.parametrize("dtype", TYPES)
def test_balance_reads_what_the_call_before_wrote(rs, dtype):
    """The scores are asked for while the expert ids are still being counted:
    they have to be those that the work queued before the call leaves."""
    tokens, experts, k = 40001, 64, 4
    g = torch.Generator(device="cuda").manual_seed(3)
    sources = [(torch.randn(tokens, experts, generator=g, device="cuda") * 2).to(dtype) for _ in range(6)]
    ids = torch.randint(0, experts, (tokens, k), generator=g, device="cuda")
    mask = torch.rand(tokens, generator=g, device="cuda") < 0.8
    up = torch.tensor([1e4], device="cuda")
    _, counts, _, n = rs.balance_loss(sources[0], ids)
    writes = [lambda to, s: to.copy_(s),
              lambda to, s: rs.balance_loss_backward(up, s, counts, n, k, grad_out=to)]
    for token_mask in (None, mask):
        for write in writes:
            want = []
            for s in sources:
                x = torch.empty_like(s)
                write(x, s)
                torch.cuda.synchronize()
                want.append(rs.balance_loss_grad(x, ids, token_mask=token_mask))
                torch.cuda.synchronize()
            x, got = torch.empty_like(sources[0]), []
            for s in sources:
                write(x, s)
                got.append(rs.balance_loss_grad(x, ids, token_mask=token_mask))
            for a, b in zip(want, got):
                assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_balance_nan_stays_in_its_gradient_row(rs):
    x, xd, g = rows_of(40, 20, torch.float32, 7)
    x[7, 3] = math.nan
    xd.copy_(x.cuda())
    ids = torch.topk(torch.randn(40, 20, generator=g), 2).indices.cuda()
    loss, counts, mean, n, grad = rs.balance_loss_grad(xd, ids)
    assert loss.isnan() and grad[7].isnan().all() and not grad[:7].isnan().any()
    assert not grad[8:].isnan().any()


def test_no_rows(rs):
    x = torch.empty(0, 50, device="cuda")
    e = torch.empty(0, device="cuda")
    out = rs.distill_loss_grad(x, torch.empty(0, 3, device="cuda"),
                               torch.empty(0, 3, dtype=torch.int64, device="cuda"))
    assert out[0].shape == (0,) and out[2].shape == (0, 50)
    out = rs.policy_loss(x, torch.empty(0, dtype=torch.int64, device="cuda"), e, e)
    assert out[0].shape == (0,)


def test_offsets_past_32_bits(rs):
    """Rows that begin beyond 2^32 bytes and 2^31 elements of their buffer."""
    cols, stride, rows = 1000, (1 << 30) + 8, 4
    buf = torch.empty((rows - 1) * stride + cols, dtype=torch.bfloat16, device="cuda")
    x = (torch.randn(rows, cols, generator=torch.Generator().manual_seed(1)) * 3).to(torch.bfloat16)
    xd = buf.as_strided((rows, cols), (stride, 1))
    xd.copy_(x.cuda())
    values, indices = torch.topk(x, 5, dim=1)
    check_distill(rs, x, xd, values, indices)
    check_distill(rs, x, xd, values, indices, grad_out=xd)
    xd.copy_(x.cuda())
    ids = torch.topk(x[:, :64].float(), 2).indices
    check_balance(rs, x[:, :64], xd[:, :64], ids)
