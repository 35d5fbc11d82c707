"""The losses over rows of scores, as measured workloads.

Three operators, each forward ("fwd": the losses), backward ("bwd": the
gradient from saved statistics) and in one call ("grad": losses and gradient):

  distill  the KL divergence of a student's rows of logits from a teacher's
           top logits (values and column indices, as a descending row sort
           returns them), truncated to at most k per row
  policy   the clipped policy-gradient loss with a KL term to a reference
           policy, of one taken action (token) per row of logits
  balance  a router's load-balancing loss and its per-expert token counts

`own` selects the package's kernels; otherwise `run` computes the same in
elementary torch operations, in 32 bits, rounded once at the end.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f16": 2, "f32": 4}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # a few decoded positions of a small vocabulary: latency of one call
        _distill("distill_grad_bf16_8x32000_k16", "grad", "bf16", 8, 32000, 16, masked=0),
        # one training micro-batch over a large vocabulary: the largest call
        _distill("distill_grad_bf16_4096x131072_k64", "grad", "bf16", 4096, 131072, 64),
        # evaluation of a student on the row-sort shape (no gradient)
        _distill("distill_fwd_f16_1024x65536_k32", "fwd", "f16", 1024, 65536, 32, masked=0),
        # the backward call of a training graph, 32-bit logits, an odd
        # vocabulary in rows padded to a multiple of 64, temperature 2
        _distill("distill_bwd_f32_1021x50001_k33", "bwd", "f32", 1021, 50001, 33, stride=50048,
                 temperature=2.0),
        # one token of a reward-tuned answer: latency
        _policy("policy_grad_bf16_1x65536", "grad", "bf16", 1, 65536, masked=0),
        # one packed batch of answers, an eighth of the tokens being prompts
        _policy("policy_grad_bf16_8192x65536", "grad", "bf16", 8192, 65536, masked=1024),
        # log-probabilities and losses of a sampled batch, no gradient
        _policy("policy_fwd_bf16_2048x131072", "fwd", "bf16", 2048, 131072, masked=256),
        # backward over an odd vocabulary: no row but the first is aligned
        _policy("policy_bwd_f16_777x100003", "bwd", "f16", 777, 100003, masked=97),
        # a router's loss over one short sequence: latency
        _balance("balance_grad_bf16_32x8_k2", "grad", "bf16", 32, 8, 2),
        # a router with many experts over a large batch of tokens
        _balance("balance_grad_bf16_262144x256_k8", "grad", "bf16", 262144, 256, 8),
        # the same loss as a running figure, 32-bit scores, padded tokens
        _balance("balance_fwd_f32_65536x64_k4", "fwd", "f32", 65536, 64, 4, masked=8192),
        # backward, an expert count that is no power of two, an odd batch
        _balance("balance_bwd_f16_32767x160_k6", "bwd", "f16", 32767, 160, 6, masked=4095),
    ]


def _distill(name, way, dtype, rows, cols, k, stride=0, temperature=1.0, masked=None):
    return {"name": name, "op": "distill", "way": way, "dtype": dtype, "rows": rows, "cols": cols,
            "k": k, "stride": stride or cols, "temperature": temperature,
            "masked": rows // 8 if masked is None else masked}


def _policy(name, way, dtype, rows, cols, stride=0, temperature=1.0, masked=0):
    return {"name": name, "op": "policy", "way": way, "dtype": dtype, "rows": rows, "cols": cols,
            "stride": stride or cols, "temperature": temperature, "masked": masked}


def _balance(name, way, dtype, rows, cols, k, masked=0):
    return {"name": name, "op": "balance", "way": way, "dtype": dtype, "rows": rows, "cols": cols,
            "k": k, "masked": masked}


def _log_uniform(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("distill", "policy", "balance"))
    way = rng.choice(("fwd", "bwd", "grad"))
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    if op == "balance":
        cols = _log_uniform(rng, 4, 512)
        rows = _log_uniform(rng, 1, 262144)
        case = _balance("", way, dtype, rows, cols, rng.randint(1, min(8, cols)),
                        masked=rng.choice((0, rows // 8)))
    else:
        cols = _log_uniform(rng, 2000, 200000)
        most = min(8192, (1 << 28) // cols)
        rows = _log_uniform(rng, 1, most)
        stride = rng.choice((cols, cols, -(-cols // 64) * 64, cols + rng.randint(1, 9)))
        temperature = rng.choice((1.0, 1.0, 0.7, 2.0))
        masked = rng.choice((0, rows // 8))
        if op == "distill":
            case = _distill("", way, dtype, rows, cols, _log_uniform(rng, 1, 256), stride,
                            temperature, masked)
        else:
            case = _policy("", way, dtype, rows, cols, stride, temperature, masked)
    del case["name"]
    return case


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    """The tensors a training step has in hand: logits as the model's last
    product leaves them (spread about 2.5, a few columns far above the rest),
    the targets, and for the backward call the upstream gradient and the
    statistics that the forward call returned."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    rows, cols, dtype = case["rows"], case["cols"], _TYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    if case["op"] == "balance":
        lean = randn(cols) * 0.5  # some experts are liked more than others
        logits = (randn(rows, cols) * 1.5 + lean).to(dtype)
        ids = torch.topk(logits, case["k"], dim=1).indices
        # the loss's share of the objective, times the loss scale that 16-bit
        # IEEE gradients are trained with
        scale = 0.01 * (65536.0 if case["dtype"] == "f16" else 1.0)
        state = {"case": case, "logits": logits, "ids": ids, "mask": None, "scale": scale}
        if case["masked"]:
            keep = torch.ones(rows, dtype=torch.bool, device=dev)
            keep[torch.randperm(rows, generator=gen, device=dev)[:case["masked"]]] = False
            state["mask"] = keep
        if case["way"] == "bwd":
            keep = torch.ones(rows, dtype=torch.bool, device=dev) if state["mask"] is None else state["mask"]
            chosen = torch.where(keep[:, None], ids, torch.full_like(ids, cols))
            state["counts"] = torch.bincount(chosen.reshape(-1), minlength=cols + 1)[:cols].to(torch.int32)
            state["tokens"] = keep.sum().to(torch.int32).reshape(1)
            state["grad_loss"] = torch.full((1,), scale, device=dev) * (1 + torch.rand(1, generator=gen, device=dev))
        return state

    stride = case["stride"]
    buffer = torch.empty(rows, stride, dtype=dtype, device=dev)
    block = max(1, (1 << 27) // stride)
    for r in range(0, rows, block):
        n = min(block, rows - r)
        buffer[r:r + n] = randn(n, stride).mul_(2.5).to(dtype)
    logits = buffer[:, :cols]
    favoured = torch.randint(0, cols, (rows, 8), generator=gen, device=dev)
    logits.scatter_add_(1, favoured, (torch.rand(rows, 8, generator=gen, device=dev) * 12).to(dtype))
    weights = torch.ones(rows, device=dev)
    if case["masked"]:
        weights[torch.randperm(rows, generator=gen, device=dev)[:case["masked"]]] = 0.0
    weights *= (1024.0 if case["dtype"] == "f16" else 1.0) / max(1, rows - case["masked"])
    state = {"case": case, "logits": logits, "weights": weights, "temperature": case["temperature"]}

    if case["op"] == "distill":
        k = case["k"]
        values = torch.empty(rows, k, dtype=dtype, device=dev)
        indices = torch.empty(rows, k, dtype=torch.int64, device=dev)
        for r in range(0, rows, block):
            n = min(block, rows - r)
            teacher = (logits[r:r + n].float() + randn(n, cols) * 0.7).to(dtype)
            values[r:r + n], indices[r:r + n] = torch.topk(teacher, k, dim=1)
        # the teacher's list ends earlier in rows that few tokens dominate
        length = torch.randint(max(1, k // 2), k + 1, (rows, 1), generator=gen, device=dev)
        indices.masked_fill_(torch.arange(k, device=dev) >= length, -1)
        state |= {"top_values": values, "top_indices": indices}
    else:
        actions = torch.empty(rows, dtype=torch.int64, device=dev)
        logprobs = torch.empty(rows, device=dev)
        for r in range(0, rows, block):
            n = min(block, rows - r)
            x = logits[r:r + n].float() / case["temperature"]
            lse = torch.logsumexp(x, 1)
            # a sampled token: one of the row's likely ones
            pick = torch.randint(0, 8, (n, 1), generator=gen, device=dev)
            actions[r:r + n] = favoured[r:r + n].gather(1, pick)[:, 0]
            logprobs[r:r + n] = x.gather(1, actions[r:r + n, None])[:, 0] - lse
        state |= {"actions": actions, "old": logprobs + randn(rows) * 0.15,
                  "ref": logprobs + randn(rows) * 0.3, "advantages": randn(rows),
                  "clip_low": 0.2, "clip_high": 0.28, "kl_coef": 0.05}
    if case["way"] == "bwd":
        lse = torch.empty(rows, device=dev)
        for r in range(0, rows, block):
            n = min(block, rows - r)
            lse[r:r + n] = torch.logsumexp(logits[r:r + n].float() / case["temperature"], 1)
        state["lse"] = torch.where(weights == 0, torch.zeros_like(lse), lse)
        state["grad_losses"] = torch.full((rows,), 1.0, device=dev) + 0.1 * randn(rows)
    return state


# --------------------------------------------------------------- one pass
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import lsd_radix_sort_gb300 as rs
    case = s["case"]
    op, way = case["op"], case["way"]
    if op == "balance":
        if way == "fwd":
            return rs.balance_loss(s["logits"], s["ids"], token_mask=s["mask"])
        if way == "grad":
            return rs.balance_loss_grad(s["logits"], s["ids"], token_mask=s["mask"], scale=s["scale"])
        return rs.balance_loss_backward(s["grad_loss"], s["logits"], s["counts"], s["tokens"],
                                        top_k=case["k"], token_mask=s["mask"])
    if op == "distill":
        args = (s["top_values"], s["top_indices"])
        kw = {"temperature": s["temperature"], "weights": s["weights"]}
        if way == "fwd":
            return rs.distill_loss(s["logits"], *args, **kw)
        if way == "grad":
            return rs.distill_loss_grad(s["logits"], *args, **kw)
        return rs.distill_loss_backward(s["grad_losses"], s["logits"], s["lse"], *args, **kw)
    args = (s["actions"], s["old"], s["advantages"])
    kw = {"ref_logprobs": s["ref"], "clip_low": s["clip_low"], "clip_high": s["clip_high"],
          "kl_coef": s["kl_coef"], "temperature": s["temperature"], "weights": s["weights"]}
    if way == "fwd":
        return rs.policy_loss(s["logits"], *args, **kw)
    if way == "grad":
        return rs.policy_loss_grad(s["logits"], *args, **kw)
    return rs.policy_loss_backward(s["grad_losses"], s["logits"], s["lse"], *args, **kw)


def _run_plain(s):
    return {"distill": _plain_distill, "policy": _plain_policy, "balance": _plain_balance}[s["case"]["op"]](s)


def _plain_distill(s):
    x, tau, w, way = s["logits"], s["temperature"], s["weights"], s["case"]["way"]
    live = (s["top_indices"] >= 0) & (s["top_indices"] < x.shape[1])
    at = torch.where(live, s["top_indices"], torch.zeros_like(s["top_indices"]))
    t = torch.where(live, s["top_values"].float() / tau, torch.full_like(at, -math.inf, dtype=torch.float32))
    t = t - t.amax(1, keepdim=True)
    logp = t - t.exp().sum(1, keepdim=True).log()
    p = torch.where(live, logp.exp(), torch.zeros_like(logp))
    z = x.float() / tau
    out = []
    if way != "bwd":
        m = z.amax(1, keepdim=True)
        e = (z - m).exp()
        total = e.sum(1, keepdim=True)
        lse = (m + total.log())[:, 0]
        logq = z.gather(1, at) - lse[:, None]
        loss = torch.where(live, p * (logp - logq), torch.zeros_like(p)).sum(1)
        on = w != 0
        out = [torch.where(on, tau * tau * w * loss, torch.zeros_like(loss)),
               torch.where(on, lse, torch.zeros_like(lse))]
        if way == "fwd":
            return tuple(out)
        q, c = e / total, w * tau
    else:
        q, c = (z - s["lse"][:, None]).exp(), w * tau * s["grad_losses"]
    grad = q.scatter_add(1, at, -p) * c[:, None]
    grad = torch.where((w != 0)[:, None], grad, torch.zeros_like(grad)).to(x.dtype)
    return grad if way == "bwd" else (*out, grad)


def _plain_policy(s):
    x, tau, w, way = s["logits"], s["temperature"], s["weights"], s["case"]["way"]
    on = w != 0
    a = s["actions"][:, None]
    z = x.float() / tau
    if way == "bwd":
        lse = s["lse"]
    else:
        m = z.amax(1, keepdim=True)
        e = (z - m).exp()
        total = e.sum(1, keepdim=True)
        lse = (m + total.log())[:, 0]
    logp = z.gather(1, a)[:, 0] - lse
    adv = s["advantages"]
    ratio = (logp - s["old"]).exp()
    low, high = 1 - s["clip_low"], 1 + s["clip_high"]
    d = s["ref"] - logp
    zero = torch.zeros_like(logp)
    out = []
    if way != "bwd":
        surrogate = torch.minimum(ratio * adv, ratio.clamp(low, high) * adv)
        loss = w * (s["kl_coef"] * (d.exp() - d - 1) - surrogate)
        out = [torch.where(on, loss, zero), torch.where(on, logp, zero), torch.where(on, lse, zero)]
        if way == "fwd":
            return tuple(out)
    held = ((adv > 0) & (ratio > high)) | ((adv < 0) & (ratio < low))
    g = torch.where(held, zero, -adv * ratio) + s["kl_coef"] * (1 - d.exp())
    c = g * w / tau if way == "grad" else g * w * s["grad_losses"] / tau
    q = e / total if way == "grad" else (z - lse[:, None]).exp()
    grad = q * -c[:, None]
    grad = grad.scatter_add(1, a, c[:, None])
    grad = torch.where(on[:, None], grad, torch.zeros_like(grad)).to(x.dtype)
    return grad if way == "bwd" else (*out, grad)


def _plain_balance(s):
    x, mask, way, k = s["logits"], s["mask"], s["case"]["way"], s["case"]["k"]
    experts = x.shape[1]
    z = x.float()
    e = (z - z.amax(1, keepdim=True)).exp()
    p = e / e.sum(1, keepdim=True)
    if mask is not None:
        p = torch.where(mask[:, None], p, torch.zeros_like(p))
    if way == "bwd":
        counts, tokens, scale = s["counts"], s["tokens"], s["grad_loss"]
    else:
        ids = s["ids"] if mask is None else torch.where(mask[:, None], s["ids"], torch.full_like(s["ids"], experts))
        counts = torch.zeros(experts + 1, dtype=torch.int32, device=x.device)
        counts.scatter_add_(0, ids.reshape(-1), torch.ones_like(ids, dtype=torch.int32).reshape(-1))
        counts = counts[:experts]
        if mask is None:
            tokens = torch.full((1,), x.shape[0], dtype=torch.int32, device=x.device)
        else:
            tokens = mask.sum(dtype=torch.int32).reshape(1)
        scale = s["scale"]
    n = tokens.float().clamp(min=1)
    share = counts.float() * experts / (k * n)
    if way == "bwd":
        return ((share - (p * share).sum(1, keepdim=True)) * p * (scale / n)).to(x.dtype)
    mean = p.sum(0) / n
    out = ((share * mean).sum(), counts, mean, tokens)
    if way == "fwd":
        return out
    return (*out, ((share - (p * share).sum(1, keepdim=True)) * p * (scale / n)).to(x.dtype))


# ------------------------------------------------------- the least of work
def work(case):
    """Logits and targets of the rows that count read once, outputs written
    once (gradients of masked rows are zeros, written too)."""
    rows, cols, es, way = case["rows"], case["cols"], _BYTES[case["dtype"]], case["way"]
    live = rows - case["masked"]
    read = live * cols * es
    write = 0 if way == "fwd" else rows * cols * es
    flops = live * cols * {"fwd": 4, "bwd": 4, "grad": 8}[way]
    if case["op"] == "balance":
        small = (0 if way == "bwd" else live * case["k"] * 8) + (rows if case["masked"] else 0) + cols * 8
        flops += live * cols * 2
    elif case["op"] == "distill":
        small = live * case["k"] * (es + 8) + rows * 12
        flops += live * case["k"] * 8
    else:
        small = live * 24 + rows * 16
    return {"bytes": read + write + small, "flops": flops}


# ------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """The same outputs from the definitions, in 64 bits, block by block."""
    s = prepare(case, seed)
    if case["op"] == "balance":
        return _exact_balance(case, s)
    rows, cols = case["rows"], case["cols"]
    block = max(1, (1 << 26) // cols)
    parts = [_exact_rows(case, s, slice(r, min(rows, r + block))) for r in range(0, rows, block)]
    out = tuple(torch.cat(p) if p[0] is not None else None for p in zip(*parts))
    if case["way"] == "bwd":
        return out[-1]
    return out if case["way"] == "grad" else out[:-1]


def _exact_rows(case, s, at):
    tau = case["temperature"]
    z = s["logits"][at].double() / tau
    w = s["weights"][at].double()
    off = w == 0
    logq = torch.log_softmax(z, 1)
    lse = torch.logsumexp(z, 1)
    up = w * s["grad_losses"][at].double() if case["way"] == "bwd" else w
    if case["op"] == "distill":
        i = s["top_indices"][at]
        gone = (i < 0) | (i >= case["cols"])
        i = i.clamp(0, case["cols"] - 1)
        logp = torch.log_softmax((s["top_values"][at].double() / tau).masked_fill(gone, -math.inf), 1)
        p = logp.exp()
        loss = w * tau ** 2 * (p * (logp - logq.gather(1, i))).masked_fill(gone, 0).sum(1)
        firsts = (loss.masked_fill(off, 0), lse.masked_fill(off, 0))
        if case["way"] == "fwd":
            return (*firsts, None)
        grad = logq.exp_().scatter_add_(1, i, -p).mul_(tau * up[:, None])
    else:
        a = s["actions"][at][:, None]
        logp = logq.gather(1, a)[:, 0]
        adv = s["advantages"][at].double()
        old, ref = s["old"][at].double(), s["ref"][at].double()
        logp.requires_grad_(True)
        with torch.enable_grad():
            r = torch.exp(logp - old)
            gain = torch.minimum(r * adv, torch.clamp(r, 1 - s["clip_low"], 1 + s["clip_high"]) * adv)
            loss = -gain + s["kl_coef"] * (torch.expm1(ref - logp) - (ref - logp))
            g, = torch.autograd.grad(loss.sum(), logp)
        loss, logp = loss.detach(), logp.detach()
        firsts = ((w * loss).masked_fill(off, 0), logp.masked_fill(off, 0), lse.masked_fill(off, 0))
        if case["way"] == "fwd":
            return (*firsts, None)
        c = (up * g / tau)[:, None]
        grad = logq.exp_().neg_().mul_(c).scatter_add_(1, a, c)
    return (*firsts, grad.masked_fill_(off[:, None], 0))


def _exact_balance(case, s):
    x, mask = s["logits"].double(), s["mask"]
    tokens, experts = x.shape
    mask = torch.ones(tokens, dtype=torch.bool, device=x.device) if mask is None else mask
    p = torch.softmax(x, 1) * mask[:, None]
    n = max(int(mask.sum()), 1)
    counts = torch.bincount(s["ids"][mask].reshape(-1), minlength=experts)
    share = counts.double() * experts / (case["k"] * n)
    scale = s["grad_loss"].double() if case["way"] == "bwd" else s["scale"]
    grad = p * (share - (p @ share)[:, None]) * (scale / n)
    if case["way"] == "bwd":
        return grad
    mean = p.sum(0) / n
    out = ((share @ mean), counts.to(torch.int32), mean, mask.sum().to(torch.int32).reshape(1))
    return out if case["way"] == "fwd" else (*out, grad)
