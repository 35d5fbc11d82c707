"""Sorts and losses together: a small mixture-of-experts student.

    python examples/train_step.py [--steps N]

1. The teacher's rows of logits are sorted once, descending; the first k
   values and columns of each row, as they lie there, are what the student is
   distilled from (distill_loss).
2. The router's scores are sorted the same way; the first two columns are each
   token's experts.  balance_loss counts the tokens per expert, and a key-value
   sort of the (expert, slot) pairs brings each expert's tokens together: the
   counts are the lengths of its segments.
3. Then the student samples answers from its own rows, and policy_loss raises
   the probability of those that the teacher would have given, held near the
   distilled student by the KL term.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import lsd_radix_sort_gb300 as rs  # noqa: E402

TOKENS, WIDTH, VOCAB, EXPERTS, TOP_K, LIST = 512, 64, 2000, 8, 2, 32


class Student(torch.nn.Module):
    def __init__(self, gen):
        super().__init__()

        def weights(*shape):
            drawn = torch.randn(*shape, generator=gen, device="cuda")
            return torch.nn.Parameter(drawn * WIDTH ** -0.5)

        self.router = weights(WIDTH, EXPERTS)
        self.experts = weights(EXPERTS, WIDTH, WIDTH)
        self.head = weights(WIDTH, VOCAB)

    def forward(self, x, keep):
        """(logits, balance loss, counts) of the tokens x."""
        scores = x @ self.router
        ids = rs.segmented_sort(scores.detach().bfloat16(), descending=True)[1][:, :TOP_K]
        balance, counts, _, _ = rs.balance_loss(scores, ids, token_mask=keep)
        # the kept tokens' slots in expert order: padded ones sort behind the last
        experts = torch.where(keep[:, None], ids, EXPERTS).int().reshape(-1)
        slots = torch.arange(experts.numel(), dtype=torch.int32, device=x.device)
        _, order = rs.radix_sort_pairs(experts, slots, end_bit=EXPERTS.bit_length())
        gates = scores.gather(1, ids).softmax(1).reshape(-1)
        out = x.clone()
        begin = 0
        for expert, n in enumerate(counts.tolist()):
            at = order[begin:begin + n].long()
            begin += n
            token = at // TOP_K
            done = torch.tanh(x[token] @ self.experts[expert])
            out = out.index_add(0, token, done * gates[at, None])
        return out @ self.head, balance, counts


def main(steps=30, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(TOKENS, WIDTH, generator=gen, device="cuda")
    keep = torch.ones(TOKENS, dtype=torch.bool, device="cuda")
    keep[-TOKENS // 8:] = False  # padding
    weights = keep.float() / keep.sum()
    teacher = (x @ torch.randn(WIDTH, VOCAB, generator=gen, device="cuda") * 0.5).bfloat16()
    values, columns = rs.segmented_sort(teacher, descending=True)
    student = Student(gen)
    optimizer = torch.optim.Adam(student.parameters(), lr=5e-3)

    history = {"distill": [], "balance": [], "reward": []}
    for _ in range(steps):
        logits, balance, counts = student(x, keep)
        losses, _ = rs.distill_loss(logits, values[:, :LIST], columns[:, :LIST], 2.0, weights)
        assert int(counts.sum()) == int(keep.sum()) * TOP_K
        optimizer.zero_grad()
        (losses.sum() + 0.01 * balance).backward()
        optimizer.step()
        history["distill"].append(losses.sum().item())
        history["balance"].append(balance.item())

    with torch.no_grad():
        reference = student(x, keep)[0].log_softmax(1)
    optimizer = torch.optim.Adam(student.parameters(), lr=1e-3)
    for _ in range(steps):
        with torch.no_grad():
            old = student(x, keep)[0].log_softmax(1)
            actions = torch.multinomial(old.exp(), 1, generator=gen)
            reward = (columns[:, :LIST] == actions).any(1).float()
        history["reward"].append((reward * weights).sum().item())
        advantages = reward - (reward * weights).sum()
        for _ in range(4):  # passes over the same answers: ratios leave 1, clips hold
            logits, balance, _ = student(x, keep)
            losses, _, _ = rs.policy_loss(
                logits, actions[:, 0], old.gather(1, actions)[:, 0].contiguous(), advantages,
                reference.gather(1, actions)[:, 0].contiguous(), kl_coef=0.02, weights=weights)
            optimizer.zero_grad()
            (losses.sum() + 0.01 * balance).backward()
            optimizer.step()
    return history


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    parser.add_argument("--steps", type=int, default=30)
    got = main(parser.parse_args().steps)
    for name, series in got.items():
        print(f"{name}: {series[0]:.4f} -> {series[-1]:.4f}")
