"""The row losses in 64 bits on the GPU, whole matrices at a time, with bounds
that follow from the distance of each score to its row's largest and not from
the scores' size: a constant row has uniform probabilities however large its
scores, and a bound that grows with them would accept anything there."""
import math

import numpy as np
import torch

from tests.loss_oracle import ROUND, U32

# How far (in nats) a kernel's origin may lie below the row's maximum.
LAG = 30 * math.log(2.0)


class Rows:
    """The softmax of rows of scores, and the relative error that 32 bits cost a
    probability: the exponent (its product with the rounded scale, and its own
    rounding: 2 D, D being the distance to the maximum in nats; for terms of
    the sum the mean distance, which entropy bounds by log cols), the part of a
    bit per 2^24 by which a large origin's product is rounded, the additions (a
    thread's chain of at most cols / 1024, with 512 threads and two pairs of
    sums, or 16), and 96 for exponentials of 2 ulp, their repair, joins and the
    division."""

    def __init__(self, x, tau):
        self.tau = float(np.float32(tau))  # as the kernels get it
        self.z = x.double() / self.tau
        self.top = self.z.amax(1, keepdim=True)
        self.dist = torch.where(self.z == -math.inf, torch.full_like(self.z, math.inf), self.top - self.z)
        e = (-self.dist).exp()
        total = e.sum(1, keepdim=True)
        self.q = e / total
        self.log_sum = total.log()[:, 0]
        self.lse = self.top[:, 0] + self.log_sum
        cols = x.shape[1]
        self.off = (self.top[:, 0].abs() * 1.5 * 2.0 ** -24).clamp(max=64)
        self.sum_error = U32 * (2 * (math.log(cols) + LAG) + self.off + cols / 1024 + 96)

    def saved_error(self):
        """What a saved lse adds to a probability of the backward call: its own
        rounding, and that of the scores' products, where it is below 1024;
        the statistics of other rows are taken again."""
        near = self.lse.abs() < 1100
        return torch.where(near, U32 * 6 * self.lse.abs(), torch.zeros_like(self.lse))

    def q_error(self):
        return self.sum_error[:, None] + U32 * 2 * self.dist.clamp(max=200)

    def lse_error(self):
        return self.sum_error + U32 * (4 * self.lse.abs() + 2 * LAG)

    def least(self, c):
        """Probabilities that a large origin may lose."""
        return torch.where(self.off > 0.5, c.abs() * 2.0 ** -58, torch.zeros_like(c))[:, None]


def dev64(t, rows):
    return torch.ones(rows, dtype=torch.float64, device="cuda") if t is None else t.double()


def within(got, want, bound, what):
    got, want = got.double(), want.double()
    bound = bound.expand_as(want)
    same = (got == want) | (got.isnan() & want.isnan())
    far = ~(same | ((got - want).abs() <= bound))
    if bool(far.any()):
        i = tuple(int(v) for v in far.nonzero()[0])
        raise AssertionError(f"{what}: {int(far.sum())} of {far.numel()} values off, first at {i}: "
                             f"got {got[i]}, expected {want[i]}, bound {bound[i]}")


def distill(rows, x, values, indices, weights=None, up=None):
    """(losses, bound, gradient, bound, what the backward call adds to that) of
    a distillation; every row has a live entry of finite value on a column of
    finite score."""
    n, cols = x.shape
    tau, w = rows.tau, dev64(weights, n)
    live = (indices >= 0) & (indices < cols)
    at = indices.clamp(0, cols - 1).long()
    v = torch.where(live, values.double(), torch.full_like(at, -math.inf, dtype=torch.float64))
    far_v = torch.where(live, (v.amax(1, keepdim=True) - v) / tau, torch.full_like(v, math.inf))
    e = (-far_v).exp()
    log_sum_p = e.sum(1, keepdim=True).log()
    p = e / e.sum(1, keepdim=True)
    p_error = U32 * (2 * far_v.clamp(max=200) + 64 + v.shape[1] / 16)
    dist = rows.dist.gather(1, at)
    kl = torch.where(p == 0, torch.zeros_like(p), p * (-far_v - log_sum_p + dist + rows.log_sum[:, None])).sum(1)
    losses = w * tau * tau * kl
    nearest = torch.where(live, dist, torch.full_like(dist, math.inf)).amin(1, keepdim=True)
    sizes = torch.where(p == 0, torch.zeros_like(p),
                        p * (far_v + log_sum_p.abs() + dist - nearest)).sum(1) + nearest[:, 0] + rows.log_sum
    spread = torch.where(p == 0, torch.zeros_like(p), p * p_error * (far_v + dist + log_sum_p.abs())).sum(1)
    loss_bound = (w.abs() * tau * tau * (8 * U32 * (sizes + 2 * LAG) + rows.sum_error + 64 * U32 + spread)
                  + 1e-42)
    c = w * tau * dev64(up, n)
    target = torch.zeros_like(rows.z).scatter_add_(1, at, torch.where(live, p, torch.zeros_like(p)))
    target_error = torch.zeros_like(rows.z).scatter_add_(1, at, torch.where(live, p * p_error, torch.zeros_like(p)))
    grad = c[:, None] * (rows.q - target)
    u, tiny = ROUND[x.dtype]
    bound = (c.abs()[:, None] * (rows.q * rows.q_error() + target_error + 4 * U32 * (rows.q + target))
             + grad.abs() * u * 1.01 + tiny + rows.least(c))
    saved = c.abs()[:, None] * rows.q * rows.saved_error()[:, None]
    return losses, loss_bound, grad, bound, saved


def policy(rows, x, actions, old, adv, ref=None, low=0.2, high=0.28, kl=0.0, weights=None, up=None):
    """(losses, bound, log-probabilities, bound, gradient, bound, what the
    backward call adds to that)."""
    n = x.shape[0]
    w, adv, old = dev64(weights, n), adv.double(), old.double()
    a = actions.long()[:, None]
    dist = rows.dist.gather(1, a)[:, 0]
    logp = -dist - rows.log_sum
    logp_error = U32 * 4 * (dist + LAG + rows.log_sum) + rows.sum_error
    exponent_error = logp_error + U32 * 4 * (logp.abs() + old.abs() + 4)
    ratio = (logp - old).exp()
    held = ((adv > 0) & (ratio > 1 + high)) | ((adv < 0) & (ratio < 1 - low))
    loss = -torch.minimum(ratio * adv, ratio.clamp(1 - low, 1 + high) * adv)
    g = torch.where(held, torch.zeros_like(ratio), -adv * ratio)
    size = (adv * ratio).abs()
    if kl:
        d = ref.double() - logp
        loss = loss + kl * (torch.expm1(d) - d)
        g = g - kl * torch.expm1(d)
        exponent_error = exponent_error + U32 * 4 * ref.double().abs()
        size = size + abs(kl) * (1 + d.exp()) * (1 + d.abs())
    loss_bound = w.abs() * size * (2 * exponent_error + 32 * U32)
    c = w * dev64(up, n) * g / rows.tau
    c_bound = (w * dev64(up, n)).abs() / rows.tau * size * (2 * exponent_error + 32 * U32)
    taken = torch.zeros_like(rows.z).scatter_(1, a, 1.0)
    grad = c[:, None] * (taken - rows.q)
    u, tiny = ROUND[x.dtype]
    bound = (c_bound[:, None] * (taken + rows.q) + c.abs()[:, None] * rows.q * rows.q_error()
             + 4 * U32 * c.abs()[:, None] * (rows.q + taken) + grad.abs() * u * 1.01 + tiny + rows.least(c))
    more = (rows.saved_error() + 4 * U32 * dist.clamp(max=1e4))[:, None]
    saved = ((w * dev64(up, n)).abs() / rows.tau * size)[:, None] * 2 * more * (taken + rows.q)
    saved = saved + c.abs()[:, None] * rows.q * more
    return w * loss, loss_bound, logp, logp_error, grad, bound, saved
