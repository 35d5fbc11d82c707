"""The vocabulary's two ends with the losses and the sorts, as a training step
uses them, and the example that does."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


def close(got, want, terms, what):
    """Norm-wise: sums of `terms` terms in 32 bits, one after another, lose
    2^-24 of their size per term at most."""
    error = (got.double() - want).norm() / want.norm()
    assert error <= terms * 2.0 ** -24, f"{what}: {float(error)} of {terms * 2.0 ** -24}"


def test_a_step_of_all_of_them(rs):
    """Words to rows, a layer, and back to words: distillation on lists that
    token_logprobs made, the policy loss on its log probabilities, an entropy
    bonus, a penalty on the log-sum-exp, and the likelihood of given words."""
    tokens, words, width, vocab = 300, 90, 48, 1500
    g = torch.Generator("cuda").manual_seed(1)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    ids = torch.randint(0, words, (tokens,), generator=g, device="cuda")
    ids[::7] = -1
    table, head = randn(words, width), randn(width, vocab) * width ** -0.5
    teacher = rs.token_logprobs(randn(tokens, vocab) * 3, top=24)
    taken = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    given = torch.randint(0, vocab, (tokens, 3), generator=g, device="cuda")
    advantages = randn(tokens)
    with torch.no_grad():
        start = rs.embedding(table, ids, scale=2.0) @ head
        old = rs.token_logprobs(start + 0.1 * randn(tokens, vocab), taken).logprobs
        ref = rs.token_logprobs(start + 0.2 * randn(tokens, vocab), taken).logprobs

    leaves = [table.clone().requires_grad_(True), head.clone().requires_grad_(True)]
    logits = rs.embedding(leaves[0], ids, scale=2.0) @ leaves[1]
    distill, _ = rs.distill_loss(logits, teacher.top_logprobs, teacher.top_ids, 2.0)
    policy, _, _ = rs.policy_loss(logits, taken, old, advantages, ref, kl_coef=0.1)
    made = rs.token_logprobs(logits, given, top=4, temperature=0.9)
    goal = (distill.sum() + policy.sum() - 0.01 * made.entropy.sum() + 1e-3 * (made.lse ** 2).sum()
            - made.logprobs.sum() + 0.1 * made.top_logprobs.sum())
    goal.backward()

    exact = [table.double().requires_grad_(True), head.double().requires_grad_(True)]
    rows = torch.where((ids >= 0)[:, None], exact[0][ids.clamp(min=0)] * 2.0, torch.zeros((), dtype=torch.float64, device="cuda"))
    z = rows @ exact[1]
    logq2, logq = torch.log_softmax(z / 2, 1), torch.log_softmax(z, 1)
    logp = torch.log_softmax(teacher.top_logprobs.double() / 2, 1)
    want = 4 * (logp.exp() * (logp - logq2.gather(1, teacher.top_ids))).sum()
    lp = logq.gather(1, taken[:, None])[:, 0]
    ratio, d = (lp - old).exp(), ref - lp
    adv = advantages.double()
    want = want + (-torch.minimum(ratio * adv, ratio.clamp(0.8, 1.2) * adv) + 0.1 * (torch.expm1(d) - d)).sum()
    y = z / float(torch.tensor(0.9))
    logy = torch.log_softmax(y, 1)
    want = (want + 0.01 * (logy.exp() * logy).sum() + 1e-3 * (torch.logsumexp(y, 1) ** 2).sum()
            - logy.gather(1, given).sum() + 0.1 * logy.gather(1, made.top_ids).sum())
    want.backward()
    # forward: a product over the width and sums over the vocabulary; back: one
    # over the vocabulary or the tokens, and a word's places
    terms = 2 * (width + vocab) + vocab + tokens + 256
    close(leaves[1].grad, exact[1].grad, terms, "head")
    close(leaves[0].grad, exact[0].grad, terms, "table")


def test_the_step_replays_from_a_graph(rs):
    """Lookup, scores, their gradient and the named rows' gradient, captured
    once and replayed on other words."""
    g = torch.Generator("cuda").manual_seed(2)
    table = torch.randn(5000, 64, generator=g, device="cuda").bfloat16()
    head = (torch.randn(64, 9000, generator=g, device="cuda") / 8).bfloat16()
    words = torch.randint(0, 5000, (2500,), generator=g, device="cuda")
    target = torch.randint(0, 9000, (2500,), generator=g, device="cuda")
    up = torch.full((2500,), 1 / 2500, device="cuda")

    def step():
        logits = rs.embedding(table, words, scale=8.0) @ head
        made = rs.token_logprobs(logits, target, top=5)
        back = rs.token_logprobs_backward(logits, made.stats, tokens=target, grad_logprobs=up)
        return made, rs.embedding_grad_rows(back @ head.t(), words, 5000, scale=8.0, dtype=torch.float32)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        made, (row_ids, rows, count) = step()
    for _ in range(2):
        words.copy_(torch.randint(0, 5000, (2500,), generator=g, device="cuda"))
        target.copy_(torch.randint(0, 9000, (2500,), generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        want, (want_ids, want_rows, want_count) = step()
        assert all(torch.equal(a, b) for a, b in zip(made, want))
        n = int(want_count)
        assert int(count) == n and torch.equal(row_ids, want_ids)
        assert torch.equal(rows[:n], want_rows[:n])


def test_the_example_runs_and_its_gradients_are_finite(rs):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "train_step.py")
    spec = importlib.util.spec_from_file_location("train_step_vocab", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    example.main(steps=2)
    g = torch.Generator("cuda").manual_seed(3)
    student = example.Student(g, torch.randn(example.WORDS, example.WIDTH, generator=g, device="cuda"))
    words = torch.randint(0, example.WORDS, (200,), generator=g, device="cuda")
    keep = torch.ones(200, dtype=torch.bool, device="cuda")
    logits, balance, _ = student(words, keep)
    (rs.token_logprobs(logits, words).logprobs.sum() + balance).backward()
    for name, parameter in student.named_parameters():
        assert parameter.grad is not None and parameter.grad.isfinite().all(), name
    named = torch.zeros(example.WORDS, dtype=torch.bool, device="cuda")
    named[words] = True
    assert (student.table.grad[~named] == 0).all() and student.table.grad[named].abs().sum() > 0
