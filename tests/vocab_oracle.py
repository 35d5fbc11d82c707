"""Log probabilities and embedding gradients in 64 bits, straight from their
formulas, and the bounds that the 32-bit kernels are held to."""
import math

import torch

from tests.loss_oracle import ROUND, U32

# How far (in nats) a kernel's origin may lie below the row's maximum: 2^8.
LAG = 8 * math.log(2.0)


class Logprobs:
    """Rows of scores (on any device) and what 32 bits may cost: see
    tests/loss_bounds.py for the parts of a probability's relative error.  dist
    is each score's distance to the row's largest, in nats."""

    def __init__(self, x, tau=1.0):
        self.x, self.tau = x, float(torch.tensor(tau, dtype=torch.float32))
        z = x.double() / self.tau
        self.m = x.double().amax(1)
        self.empty = self.m == -math.inf
        top = torch.where(self.empty, torch.zeros_like(self.m), z.amax(1))[:, None]
        self.dist = torch.where(z == -math.inf, torch.full_like(z, math.inf), top - z)
        e = (-self.dist).exp()
        total = e.sum(1)
        self.log_sum = total.log()
        self.q = torch.where(self.empty[:, None], torch.zeros_like(e), e / total[:, None])
        near = torch.where(self.q == 0, torch.zeros_like(self.dist), self.dist)
        mean, square = (self.q * near).sum(1), (self.q * near * near).sum(1)
        self.entropy = torch.where(self.empty, torch.zeros_like(total), self.log_sum + mean)
        self.lse = torch.where(self.empty, torch.full_like(total, -math.inf), top[:, 0] + self.log_sum)
        cols = x.shape[1]
        off = (top[:, 0].abs() * 1.5 * 2.0 ** -24).clamp(max=64)
        self.sum_error = U32 * (2 * (math.log(cols) + LAG) + off + cols / 1024 + 96)
        logs = torch.where(self.empty, torch.zeros_like(total), self.log_sum.abs())
        # errors of a term e y: e's own, y's, and those of the additions
        self.entropy_error = self.sum_error * (2 + mean + LAG) + 4 * U32 * (square + mean + LAG + logs)
        self.lse_error = self.sum_error + 4 * U32 * (top[:, 0].abs() + logs)
        self.stats_error = self.sum_error + 2 * U32 * logs
        self.logs = logs

    def logprobs(self, columns):
        """(log probabilities, bound) of columns; 0 where one is outside the row."""
        cols = self.x.shape[1]
        live = (columns >= 0) & (columns < cols)
        at = columns.long().clamp(0, cols - 1)
        dist = self.dist.gather(1, at)
        logp = torch.where(self.empty[:, None], torch.full_like(dist, -math.inf), -dist - self.log_sum[:, None])
        bound = 4 * U32 * (dist.clamp(max=1e38) + LAG + self.logs[:, None]) + self.sum_error[:, None]
        return torch.where(live, logp, torch.zeros_like(logp)), bound

    def top(self, top):
        """The columns of the best scores, -1 where there are fewer."""
        rows, cols = self.x.shape
        values, columns = torch.sort(self.x.double() + 0.0, dim=1, descending=True, stable=True)
        columns = torch.where(values == -math.inf, torch.full_like(columns, -1), columns)[:, :top]
        if top > cols:
            columns = torch.cat((columns, torch.full((rows, top - cols), -1, device=columns.device)), 1)
        return columns

    def grad(self, entries=(), g_entropy=None, g_lse=None):
        """(gradient, bound); entries: (columns, upstream gradients) pairs."""
        rows, cols = self.x.shape
        zero = torch.zeros(rows, dtype=torch.float64, device=self.x.device)
        g_h = zero if g_entropy is None else g_entropy.double()
        g_l = zero if g_lse is None else g_lse.double()
        at, size, n = torch.zeros_like(self.q), torch.zeros_like(self.q), 1
        s, s_abs = zero.clone(), zero.clone()
        for columns, g in entries:
            live = (columns >= 0) & (columns < cols)
            g = torch.where(live, g.double(), torch.zeros_like(g.double()))
            i = columns.long().clamp(0, cols - 1)
            at.scatter_add_(1, i, g)
            size.scatter_add_(1, i, g.abs())
            s, s_abs, n = s + g.sum(1), s_abs + g.abs().sum(1), n + g.shape[1]
        gone = self.empty[:, None]
        dist = torch.where(self.q == 0, torch.zeros_like(self.dist), self.dist)
        logq = -dist - torch.where(self.empty, zero, self.log_sum)[:, None]
        pull = (g_l - s)[:, None] - g_h[:, None] * (logq + self.entropy[:, None])
        grad = torch.where(gone, torch.zeros_like(at), self.q * pull + at) / self.tau
        reach = (g_l.abs() + s_abs)[:, None] + g_h.abs()[:, None] * (logq.abs() + self.entropy.abs()[:, None])
        q_error = 2 * self.sum_error[:, None] + U32 * (2 * dist + 4 * self.logs[:, None] + 16)
        log_error = (4 * U32 * (dist + LAG + self.logs[:, None]) + 2 * self.sum_error[:, None]
                     + self.entropy_error[:, None])
        u, tiny = ROUND[self.x.dtype]
        bound = (self.q * (q_error * reach + U32 * (8 + n) * 2 * reach + g_h.abs()[:, None] * log_error)
                 + U32 * (4 + n) * size) / self.tau + grad.abs() * u * 1.01 + tiny
        return grad, bound


def embedding_grad(up, ids, vocab, scale=1.0, padding_id=-1):
    """(gradient, sum of the terms' sizes, number of terms) per row of the table."""
    width = up.shape[-1]
    up, ids = up.reshape(-1, width).double(), ids.reshape(-1).long()
    live = (ids >= 0) & (ids < vocab) & (ids != padding_id)
    out = torch.zeros(vocab, width, dtype=torch.float64, device=up.device)
    size, n = out.clone(), torch.zeros(vocab, dtype=torch.float64, device=up.device)
    out.index_add_(0, ids[live], up[live])
    size.index_add_(0, ids[live], up[live].abs())
    n.index_add_(0, ids[live], torch.ones_like(ids[live], dtype=torch.float64))
    s = float(torch.tensor(scale, dtype=torch.float32))
    return out * s, size * abs(s), n


def embedding_bound(want, size, n, dtype):
    """A sum of n terms in 32 bits (n - 1 roundings at most, whatever its
    order), its product with the scale, and the rounding to the type."""
    u, tiny = ROUND[dtype]
    return U32 * (n[:, None] + 2) * size + want.abs() * u * 1.01 + tiny
