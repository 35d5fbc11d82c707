"""The order of memory operations inside one call of a loss: CTAs of a cluster
that begin apart, gradients written over the scores that others still read,
copies that overtake reads.  Each call is repeated under load and compared bit
by bit with a first one."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def rows_of(rows, cols, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(rows, cols, generator=g, device="cuda") * 3).to(dtype), g


def policy_of(x, g):
    rows, cols = x.shape
    actions = torch.randint(0, cols, (rows,), generator=g, device="cuda")
    logp = torch.log_softmax(x.float(), 1).gather(1, actions[:, None])[:, 0]
    old = logp + 0.1 * torch.randn(rows, generator=g, device="cuda")
    return actions, old, torch.randn(rows, generator=g, device="cuda")


class Load:
    """Copies on a stream of their own, which keep memory and SMs busy."""

    def __init__(self):
        self.stream = torch.cuda.Stream()
        self.a = torch.zeros(1 << 26, dtype=torch.int32, device="cuda")
        self.b = torch.empty_like(self.a)
        torch.cuda.synchronize()

    def more(self, n=1):
        with torch.cuda.stream(self.stream):
            for _ in range(n):
                self.b.copy_(self.a)


def same(a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("rows,cols", [(1, 65536), (7, 131072), (40, 50001), (70, 300000)])
def test_losses_of_clusters_that_begin_apart(rs, rows, cols):
    x, g = rows_of(rows, cols, torch.bfloat16)
    actions, old, adv = policy_of(x, g)
    values, indices = torch.topk(x, 20, dim=1)
    first = rs.policy_loss(x, actions, old, adv), rs.distill_loss(x, values, indices)
    load = Load()
    for _ in range(30):
        load.more()
        assert same(first[0], rs.policy_loss(x, actions, old, adv))
        assert same(first[1], rs.distill_loss(x, values, indices))
    torch.cuda.synchronize()


# rows too few for the SMs and rows of more than twice the ring are shared by a
# cluster; the others are a CTA's each, in registers or in the ring
IN_PLACE = [(1, 65536, torch.bfloat16), (3, 30000, torch.float16), (9, 50001, torch.float32),
            (37, 131072, torch.bfloat16), (70, 65536, torch.bfloat16), (12, 400000, torch.float32),
            (90, 400000, torch.float32), (200, 40000, torch.bfloat16), (320, 12000, torch.float32)]


@pytest.mark.parametrize("rows,cols,dtype", IN_PLACE)
def test_gradient_over_the_logits_under_load(rs, rows, cols, dtype):
    """Every CTA of a cluster reads the targets' scores of the whole row: none
    of them may be a gradient yet."""
    x, g = rows_of(rows, cols, dtype, 1)
    actions, old, adv = policy_of(x, g)
    ref = old + 0.1
    values, indices = torch.topk(x, 300, dim=1)  # a long list takes long to read
    calls = [lambda y, out: rs.policy_loss_grad(y, actions, old, adv, ref, kl_coef=0.1, grad_out=out),
             lambda y, out: rs.distill_loss_grad(y, values, indices, grad_out=out),
             lambda y, out: rs.distill_loss_grad(y, values[:, :1], indices[:, :1], grad_out=out)]
    want = [call(x, None) for call in calls]
    load, y = Load(), torch.empty_like(x)
    for _ in range(40):
        load.more()
        for call, expected in zip(calls, want):
            y.copy_(x)
            assert same(call(y, y), expected)
    torch.cuda.synchronize()


@pytest.mark.parametrize("rows,cols,dtype", IN_PLACE)
def test_backward_over_the_logits_under_load(rs, rows, cols, dtype):
    x, g = rows_of(rows, cols, dtype, 2)
    actions, old, adv = policy_of(x, g)
    values, indices = torch.topk(x, 300, dim=1)
    lse = rs.policy_loss(x, actions, old, adv)[2]
    calls = [lambda y, out: rs.policy_loss_backward(None, y, lse, actions, old, adv, grad_out=out),
             lambda y, out: rs.distill_loss_backward(None, y, lse, values, indices, grad_out=out)]
    want = [call(x, None) for call in calls]
    load, y = Load(), torch.empty_like(x)
    for _ in range(20):
        load.more()
        for call, expected in zip(calls, want):
            y.copy_(x)
            assert torch.equal(call(y, y), expected)
    torch.cuda.synchronize()


@pytest.mark.parametrize("rows,cols,dtype", [(1000, 65537, torch.bfloat16), (600, 50003, torch.float32),
                                             (1000, 70003, torch.float16)])
def test_ragged_rows_give_the_same_bits_under_load(rs, rows, cols, dtype):
    """The ends of rows that are no whole vectors are stored to their ring slots
    by a warp, and the next bulk copy lands on them."""
    x, g = rows_of(rows, cols, dtype, 3)
    actions, old, adv = policy_of(x, g)
    values, indices = torch.topk(x, 9, dim=1)
    first = rs.policy_loss_grad(x, actions, old, adv), rs.distill_loss_grad(x, values, indices)
    # the ends, against plain arithmetic: the last and first eight columns
    q = torch.softmax(x.float(), 1)
    target = torch.zeros_like(q).scatter_add_(1, indices, torch.softmax(values.float(), 1))
    for part in (slice(0, 8), slice(cols - 8, cols)):
        want = (q - target)[:, part]
        u = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 0}[dtype]
        # two 32-bit evaluations, each of at most 4e-4 relative (cols / 32 additions)
        assert bool(((first[1][2][:, part].float() - want).abs()
                     <= u * want.abs() + 8e-4 * (q + target)[:, part] + 2.0 ** -24).all())
    for _ in range(30):
        assert same(first[0], rs.policy_loss_grad(x, actions, old, adv))
        assert same(first[1], rs.distill_loss_grad(x, values, indices))


def test_balance_reads_nothing_before_its_wait():
    """The source of the balance kernel: no score and no mask byte is loaded
    ahead of the wait for what was queued before it (a prefetch to L2 is no
    read); a stale read would show only now and then."""
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                        "lsd_radix_sort_gb300", "csrc", "balance.cuh")
    with open(path) as f:
        source = f.read()
    body = source[source.index("    balance_kernel(const BalanceArgs a"):]
    before = body[:body.index("grid_dependency_sync();")]
    calls = [line for line in before.split("\n") if "load(" in line and "auto load" not in line]
    assert calls == ["        if (kept && on[u]) raw[q][u] = B::load(x + u * group * kN);"]  # load's own


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_balance_after_a_mask_was_written(rs, dtype):
    """The mask and the scores are overwritten right before each call."""
    tokens, experts, k = 50000, 64, 4
    g = torch.Generator(device="cuda").manual_seed(4)
    sources = [(torch.randn(tokens, experts, generator=g, device="cuda") * 2).to(dtype) for _ in range(5)]
    masks = [torch.rand(tokens, generator=g, device="cuda") < 0.5 for _ in range(5)]
    ids = torch.randint(0, experts, (tokens, k), generator=g, device="cuda")
    want = []
    for s, m in zip(sources, masks):
        want.append(rs.balance_loss_grad(s, ids, token_mask=m))
        torch.cuda.synchronize()
    x, mask = torch.empty_like(sources[0]), torch.empty_like(masks[0])
    for _ in range(10):
        got = []
        for s, m in zip(sources, masks):
            x.copy_(s)
            mask.copy_(m)
            got.append(rs.balance_loss_grad(x, ids, token_mask=mask))
        assert all(same(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(40, 1003), (40, 7001), (310, 9001), (310, 30003), (40, 30003), (200, 50003)])
def test_gradients_aligned_otherwise(rs, rows, cols, dtype):
    """Logits in padded rows, the gradient in packed ones and in rows that begin
    elsewhere in their 16 bytes: the bits of a gradient aligned as the logits,
    and nothing beside it is written."""
    g = torch.Generator(device="cuda").manual_seed(cols)
    wide = torch.randn(rows, cols + 21, generator=g, device="cuda").to(dtype)
    x = wide[:, :cols]
    actions = torch.randint(0, cols, (rows,), generator=g, device="cuda")
    old = torch.full((rows,), -8.0, device="cuda")
    adv = torch.randn(rows, generator=g, device="cuda")
    values, indices = torch.topk(x, 6, dim=1)
    lse = rs.policy_loss(x, actions, old, adv)[2]
    calls = [lambda out: rs.policy_loss_grad(x, actions, old, adv, grad_out=out)[3],
             lambda out: rs.distill_loss_grad(x, values, indices, grad_out=out)[2],
             lambda out: rs.policy_loss_backward(None, x, lse, actions, old, adv, grad_out=out),
             lambda out: rs.distill_loss_backward(None, x, lse, values, indices, grad_out=out)]
    for call in calls:
        like = torch.empty_like(wide)[:, :cols]
        want = call(like).clone()
        packed = call(torch.empty(rows, cols, dtype=dtype, device="cuda"))
        assert torch.equal(packed, want)
        for pad, shift in ((9, 1), (5, 3), (16, 8)):
            buf = torch.full((rows * (cols + pad) + 64,), 7.0, dtype=dtype, device="cuda")
            out = buf[shift:].as_strided((rows, cols), (cols + pad, 1), shift)
            assert torch.equal(call(out), want)
            out.fill_(7.0)
            assert bool((buf == 7.0).all())


@pytest.mark.parametrize("rows", [151, 152, 153, 160, 299, 300, 304])
def test_both_ways_of_middling_rows_agree(rs, rows):
    """Rows of 32 to 64 KB are held in registers where they outnumber the SMs,
    and in the ring otherwise: each row against the same row among few others."""
    x, g = rows_of(rows, 20000, torch.bfloat16, 5)
    actions, old, adv = policy_of(x, g)
    out = rs.policy_loss_grad(x, actions, old, adv)
    few = rs.policy_loss_grad(x[:5], actions[:5], old[:5], adv[:5])
    for a, b in zip(out, few):
        # the two ways add up in other orders: 20,000 / 32 additions, and a rounding to bf16
        u = 2.0 ** -8 if b.dtype is torch.bfloat16 else 0
        assert bool(((a[:5].double() - b.double()).abs()
                     <= b.double().abs() * (u + 1e-4) + 1e-4 * (b.dim() == 1) + 1e-9).all())
