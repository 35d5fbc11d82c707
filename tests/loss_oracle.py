"""The losses over rows of scores in 64 bits, on the CPU, straight from their
formulas, and the bounds that the 32-bit kernels are held to."""
import math

import torch

U32 = 2.0 ** -24
# unit roundoff and smallest subnormal of the types a gradient is rounded to
# (32-bit terms below the normal range may become 0)
ROUND = {torch.float16: (2.0 ** -11, 2.0 ** -24), torch.bfloat16: (2.0 ** -8, 2.0 ** -120),
         torch.float32: (U32, 2.0 ** -120)}


def softmax_rows(x, tau):
    """(z, lse, q, empty) of rows: -inf takes no part; an empty row has q = 0."""
    z = x.double() / tau
    m = z.amax(1, keepdim=True)
    empty = m[:, 0] == -math.inf
    o = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = (z - o).exp()
    s = e.sum(1, keepdim=True)
    lse = torch.where(empty, torch.full_like(m[:, 0], -math.inf), o[:, 0] + s[:, 0].log())
    return z, lse, torch.where(empty[:, None], torch.zeros_like(e), e / s), empty


def distill(x, values, indices, tau=1.0, weights=None, up=None):
    """(losses, lse, grad, scale of the gradient's terms)."""
    rows, cols = x.shape
    w = torch.ones(rows, dtype=torch.float64) if weights is None else weights.double()
    up = torch.ones(rows, dtype=torch.float64) if up is None else up.double()
    losses, lses = torch.zeros(rows, dtype=torch.float64), torch.zeros(rows, dtype=torch.float64)
    grad = torch.zeros(rows, cols, dtype=torch.float64)
    size = torch.zeros(rows, cols, dtype=torch.float64)
    for r in range(rows):
        if w[r] == 0:
            continue
        z, lse, q, empty = softmax_rows(x[r:r + 1], tau)
        lses[r] = lse
        live = (indices[r] >= 0) & (indices[r] < cols)
        t = values[r][live].double() / tau
        i = indices[r][live].long()
        if bool(empty) or t.numel() == 0 or bool((t == -math.inf).all()):
            continue
        logp = t - torch.logsumexp(t, 0)
        p = logp.exp()
        term = torch.where(p == 0, torch.zeros_like(p), p * (logp - (z[0, i] - lse)))
        losses[r] = w[r] * tau * tau * term.sum()
        target = torch.zeros(cols, dtype=torch.float64).index_add_(0, i, p)
        c = w[r] * up[r] * tau
        grad[r] = c * (q[0] - target)
        size[r] = c.abs() * (q[0] + target)
    return losses, lses, grad, size


def policy(x, actions, old, adv, ref=None, low=0.2, high=0.2, kl=0.0, tau=1.0, weights=None,
           up=None):
    """(losses, logprobs, lse, grad, scale of the gradient's terms, scale of the
    loss's terms); the scales bound what an error of the log-probability does."""
    rows, cols = x.shape
    w = torch.ones(rows, dtype=torch.float64) if weights is None else weights.double()
    up = torch.ones(rows, dtype=torch.float64) if up is None else up.double()
    out = [torch.zeros(rows, dtype=torch.float64) for _ in range(3)]
    grad = torch.zeros(rows, cols, dtype=torch.float64)
    size = torch.zeros(rows, cols, dtype=torch.float64)
    loss_size = torch.zeros(rows, dtype=torch.float64)
    for r in range(rows):
        a = int(actions[r])
        if w[r] == 0 or not 0 <= a < cols:
            continue
        z, lse, q, empty = softmax_rows(x[r:r + 1], tau)
        out[2][r] = lse
        logp = -math.inf if bool(empty) else float(z[0, a] - lse)
        out[1][r] = logp
        if bool(empty):
            continue
        A = float(adv[r])
        ratio = math.exp(logp - float(old[r])) if not math.isnan(logp) else math.nan
        held = (A > 0 and ratio > 1 + high) or (A < 0 and ratio < 1 - low)
        clipped = min(max(ratio, 1 - low), 1 + high)
        loss = -min(ratio * A, clipped * A)
        g = 0.0 if held else -A * ratio
        terms = abs(A) * (clipped if held else ratio)
        if kl != 0:
            d = float(ref[r]) - logp
            loss += kl * (math.exp(d) - d - 1)
            g += kl * (1 - math.exp(d))
            terms += abs(kl) * (1 + math.exp(d)) * (1 + abs(d))
        out[0][r] = w[r] * loss
        c = w[r] * up[r] * g / tau
        grad[r] = -c * q[0]
        grad[r, a] += c
        far = 1 + abs(logp) + abs(float(old[r]))
        loss_size[r] = w[r].abs() * terms * far
        size[r] = (w[r] * up[r]).abs() / tau * terms * far * q[0]
        size[r, a] += (w[r] * up[r]).abs() / tau * terms * far
    return (*out, grad, size, loss_size)


def balance(x, ids, mask=None, scale=1.0):
    """(loss, counts, mean_probs, n, grad, scale of the gradient's terms)."""
    tokens, experts = x.shape
    keep = torch.ones(tokens, dtype=torch.bool) if mask is None else mask.bool()
    p = torch.zeros(tokens, experts, dtype=torch.float64)
    if keep.any():
        p[keep] = softmax_rows(x[keep], 1.0)[2]
    chosen = ids[keep].reshape(-1).long()
    chosen = chosen[(chosen >= 0) & (chosen < experts)]
    counts = torch.bincount(chosen, minlength=experts)[:experts]
    n = max(int(keep.sum()), 1)
    share = counts.double() * experts / (ids.shape[1] * n)
    mean = p.sum(0) / n
    dot = (p @ share)[:, None]
    return (float(share @ mean), counts, mean, int(keep.sum()), scale / n * p * (share - dot),
            abs(scale) / n * p * (share + dot))


# ------------------------------------------------------------------ bounds
def row_error(x, tau):
    """Bound on the absolute error of a 32-bit lse, which is also the relative
    error of a probability: the exponent's difference and product (2 roundings
    of at most R = the row's range, which a term of weight exp(-R) carries: R
    exp(-R) < 1, so 2 roundings of min(R, 1) in the mean, and of R itself for
    one probability), the exponential (2 ulp), the sum (each thread adds its
    share of the columns one after another: at most cols / 32 of them, then
    at most 64 joins, each rescaling once), the logarithm and the last sum."""
    z = x.double() / tau
    z = torch.where(z == -math.inf, torch.full_like(z, math.nan), z)
    top = z.nan_to_num(nan=-math.inf).amax(1)
    low = z.nan_to_num(nan=math.inf).amin(1)
    span = (top - low).clamp(0, 104).nan_to_num(nan=0.0, posinf=104.0)
    size = top.abs().nan_to_num(nan=0.0, posinf=0.0, neginf=0.0)
    return U32 * (4 * span + 4 * size + x.shape[1] / 32 + 64 * 3 + 16)


def grad_bound(want, size, error, dtype):
    """Elementwise: the terms' relative errors, then one rounding to dtype."""
    u, tiny = ROUND[dtype]
    return size * (error[:, None] + 16 * U32) + want.abs() * u * 1.01 + tiny


def assert_within(got, want, bound, what):
    got, want = got.double().cpu(), want.double()
    bound = torch.as_tensor(bound, dtype=torch.float64).expand_as(want)
    same = (got == want) | (got.isnan() & want.isnan())
    far = ~(same | ((got - want).abs() <= bound))
    if far.any():
        i = tuple(int(v) for v in far.nonzero()[0])
        raise AssertionError(f"{what}: {int(far.sum())} of {far.numel()} values off, first at {i}: "
                             f"got {got[i]}, expected {want[i]}, bound {bound[i]}")
