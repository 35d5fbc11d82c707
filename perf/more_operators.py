"""The two ends of a vocabulary, as measured workloads.

  logprobs  over rows of logits: the log probabilities of given tokens, the
            row's entropy and log-sum-exp, and its top alternatives (log
            probabilities and columns); forward ("fwd") and backward ("bwd":
            the gradient from saved statistics)
  embed     the lookup of a table's rows by token, scaled ("fwd"), and its
            gradient: of the whole table ("grad"), or of the named rows only,
            in the order of their ids ("rows")

`own` selects the package's kernels; otherwise `run` computes the same in
elementary torch operations, in 32 bits, rounded once at the end.
"""
import math

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f16": 2, "f32": 4}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # the token just decoded, with what else was likely: latency of one call
        _logprobs("logprobs_fwd_bf16_1x65536_k1_top8", "fwd", "bf16", 1, 65536, 1, 8),
        # one decoding step of a batch over a large vocabulary
        _logprobs("logprobs_fwd_bf16_64x131072_k1_top20", "fwd", "bf16", 64, 131072, 1, 20),
        # every token of a long prompt scored, with alternatives: the largest call
        _logprobs("logprobs_fwd_bf16_4096x131072_k1_top20", "fwd", "bf16", 4096, 131072, 1, 20),
        # a teacher's lists for distillation, on the row-sort shape
        _logprobs("logprobs_fwd_f16_1024x65536_top64", "fwd", "f16", 1024, 65536, 0, 64),
        # four answers of a multiple choice, 32-bit logits, an odd vocabulary in
        # rows padded to a multiple of 64, sharpened
        _logprobs("logprobs_fwd_f32_1021x50001_k4", "fwd", "f32", 1021, 50001, 4, 0, 50048, 0.7),
        # policy gradient with an entropy bonus, an eighth of the tokens padded
        _logprobs("logprobs_bwd_bf16_2048x65536_k1", "bwd", "bf16", 2048, 65536, 1, 0, masked=256),
        # one decoding step of a few sequences: latency
        _embed("embed_fwd_bf16_8x131072x2048", "fwd", "bf16", 8, 131072, 2048),
        # a training batch
        _embed("embed_fwd_bf16_65536x131072x2048", "fwd", "bf16", 65536, 131072, 2048),
        # its gradient as a whole table
        _embed("embed_grad_bf16_16384x131072x2048", "grad", "bf16", 16384, 131072, 2048),
        # a padded batch into a 32-bit gradient of an odd vocabulary
        _embed("embed_grad_f16_f32_8191x50001x1000", "grad", "f16", 8191, 50001, 1000, "f32",
               masked=1024),
        # a large batch for an optimizer that updates the named rows only
        _embed("embed_rows_bf16_32768x131072x4096", "rows", "bf16", 32768, 131072, 4096),
        # the same of a short fine-tuning sequence: latency
        _embed("embed_rows_f16_512x32000x512", "rows", "f16", 512, 32000, 512),
    ]


def _logprobs(name, way, dtype, rows, cols, k, top, stride=0, temperature=1.0, masked=0):
    return {"name": name, "op": "logprobs", "way": way, "dtype": dtype, "rows": rows, "cols": cols,
            "k": k, "top": top, "stride": stride or cols, "temperature": temperature,
            "masked": masked}


def _embed(name, way, dtype, tokens, vocab, width, out=None, masked=0):
    return {"name": name, "op": "embed", "way": way, "dtype": dtype, "tokens": tokens,
            "vocab": vocab, "width": width, "out": out or dtype, "masked": masked}


def _log_uniform(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    if rng.choice(("logprobs", "embed")) == "logprobs":
        way = rng.choice(("fwd", "fwd", "bwd"))
        cols = _log_uniform(rng, 2000, 200000)
        rows = _log_uniform(rng, 1, min(4096, (1 << 28) // cols))
        stride = rng.choice((cols, cols, -(-cols // 64) * 64, cols + rng.randint(1, 9)))
        top = rng.choice((0, rng.randint(1, 20), rng.randint(1, 20), rng.randint(21, 128)))
        k = rng.choice((1, 1, rng.randint(2, 8), 0 if top else 1))
        case = _logprobs("", way, dtype, rows, cols, k, top, stride, rng.choice((1.0, 1.0, 0.7, 2.0)),
                         rng.choice((0, rows // 8)))
    else:
        way = rng.choice(("fwd", "grad", "rows"))
        width = _log_uniform(rng, 64, 8192)
        width = rng.choice((width, max(8, width // 8 * 8), -(-width // 64) * 64))
        vocab = _log_uniform(rng, 1000, min(200000, (1 << 28) // width))
        tokens = _log_uniform(rng, 1, min(65536, (1 << 27) // width))
        out = dtype if way == "fwd" else rng.choice((dtype, "f32"))
        case = _embed("", way, dtype, tokens, vocab, width, out, rng.choice((0, tokens // 8)))
    del case["name"]
    return case


# Tokens as text has them: the n-th most frequent one has a share of about
# 1 / (n + 2.7), whatever its id.
def _shares(vocab):
    p = 1.0 / (np.arange(vocab) + 2.7)
    return p / p.sum()


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    return (_prepare_embed if case["op"] == "embed" else _prepare_logprobs)(case, dev, gen)


def _prepare_logprobs(case, dev, gen):
    """Logits as a model's last product leaves them (spread about 2.5, a few
    columns far above the rest) and tokens that are likely there; for the
    backward call the upstream gradients and what the forward call returned."""
    rows, cols, stride, dtype = case["rows"], case["cols"], case["stride"], _TYPES[case["dtype"]]
    k, top, tau = case["k"], case["top"], case["temperature"]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    buffer = torch.empty(rows, stride, dtype=dtype, device=dev)
    block = max(1, (1 << 27) // stride)
    for r in range(0, rows, block):
        n = min(block, rows - r)
        buffer[r:r + n] = randn(n, stride).mul_(2.5).to(dtype)
    logits = buffer[:, :cols]
    favoured = torch.randint(0, cols, (rows, 8), generator=gen, device=dev)
    logits.scatter_add_(1, favoured, (torch.rand(rows, 8, generator=gen, device=dev) * 12).to(dtype))
    state = {"case": case, "logits": logits, "tokens": None}
    if k:
        tokens = favoured[:, :k].clone()
        if case["masked"]:  # padded positions: no token
            tokens[torch.randperm(rows, generator=gen, device=dev)[:case["masked"]]] = -1
        state["tokens"] = tokens
    if case["way"] == "bwd":
        state |= {"stats": torch.empty(rows, 2, device=dev), "entropy": torch.empty(rows, device=dev),
                  "top_ids": torch.empty(rows, top, dtype=torch.int64, device=dev) if top else None}
        for r in range(0, rows, block):
            x = logits[r:r + block].float()
            z = x / tau
            logq = torch.log_softmax(z, 1)
            state["entropy"][r:r + block] = -(logq.exp() * logq).sum(1)
            m = x.amax(1)
            state["stats"][r:r + block, 0] = m
            state["stats"][r:r + block, 1] = torch.logsumexp(z - (m / tau)[:, None], 1)
            if top:
                state["top_ids"][r:r + block] = _top(logits[r:r + block], top)[1]
        # shares of a mean over the rows, times the loss scale of 16-bit floats
        unit = (1024.0 if case["dtype"] == "f16" else 1.0) / rows
        state["grad_logprobs"] = randn(rows, k).mul_(unit) if k else None
        state["grad_entropy"] = torch.full((rows,), -0.01 * unit, device=dev)
        state["grad_lse"] = randn(rows).abs_().mul_(1e-3 * unit)
        state["grad_top"] = randn(rows, top).mul_(unit) if top else None
    return state


def _prepare_embed(case, dev, gen):
    tokens, vocab, width = case["tokens"], case["vocab"], case["width"]
    dtype, out = _TYPES[case["dtype"]], _TYPES[case["out"]]
    bounds = torch.from_numpy(np.cumsum(_shares(vocab))).to(dev)
    drawn = torch.rand(tokens, generator=gen, device=dev, dtype=torch.float64)
    nth = torch.searchsorted(bounds, drawn).clamp_(max=vocab - 1)
    ids = torch.randperm(vocab, generator=gen, device=dev)[nth]
    if case["masked"]:  # padded positions: no token
        ids[torch.randperm(tokens, generator=gen, device=dev)[:case["masked"]]] = -1
    state = {"case": case, "ids": ids, "scale": math.sqrt(width)}
    rows = vocab if case["way"] == "fwd" else tokens
    data = torch.empty(rows, width, dtype=dtype, device=dev)
    block = max(1, (1 << 27) // width)
    for r in range(0, rows, block):
        n = min(block, rows - r)
        data[r:r + n] = torch.randn(n, width, generator=gen, device=dev).mul_(0.02).to(dtype)
    state["table" if case["way"] == "fwd" else "grad"] = data
    if case["way"] == "rows":  # the optimizer's buffers: rows past the count stay as they are
        n = min(tokens, vocab)
        state["row_ids"] = torch.empty(n, dtype=torch.int64, device=dev)
        state["rows"] = torch.zeros(n, width, dtype=out, device=dev)
    return state


# --------------------------------------------------------------- one pass
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import lsd_radix_sort_gb300 as rs
    case = s["case"]
    if case["op"] == "embed":
        if case["way"] == "fwd":
            return rs.embedding(s["table"], s["ids"], scale=s["scale"])
        out = _TYPES[case["out"]]
        if case["way"] == "grad":
            return rs.embedding_grad(s["grad"], s["ids"], case["vocab"], scale=s["scale"], dtype=out)
        return rs.embedding_grad_rows(s["grad"], s["ids"], case["vocab"], scale=s["scale"],
                                      row_ids_out=s["row_ids"], rows_out=s["rows"])
    if case["way"] == "fwd":
        got = rs.token_logprobs(s["logits"], s["tokens"], top=case["top"],
                                temperature=case["temperature"])
        return tuple(t for t in got if t is not None)
    return rs.token_logprobs_backward(
        s["logits"], s["stats"], s["entropy"], tokens=s["tokens"], top_ids=s["top_ids"],
        grad_logprobs=s["grad_logprobs"], grad_entropy=s["grad_entropy"], grad_lse=s["grad_lse"],
        grad_top=s["grad_top"], temperature=case["temperature"])


def _run_plain(s):
    case = s["case"]
    if case["op"] == "logprobs":
        return (_plain_logprobs if case["way"] == "fwd" else _plain_logprobs_backward)(s)
    return {"fwd": _plain_embed, "grad": _plain_embed_grad, "rows": _plain_embed_rows}[case["way"]](s)


def _top(x, top):
    """Scores and columns of each row's largest, equal ones by column."""
    bits = (x.float() + 0.0).view(torch.int32)
    order = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long() << 32
    order |= 0xFFFFFFFF - torch.arange(x.shape[1], device=x.device)
    columns = 0xFFFFFFFF - (torch.topk(order, top, dim=1).values & 0xFFFFFFFF)
    return x.gather(1, columns).float(), columns


def _plain_logprobs(s):
    """(logprobs,) entropy, lse, (top_logprobs, top_ids,) stats"""
    x, tokens, top, tau = s["logits"], s["tokens"], s["case"]["top"], s["case"]["temperature"]
    z = x.float()
    m = z.amax(1, keepdim=True)
    y = (z - m) / tau
    e = y.exp()
    total = e.sum(1, keepdim=True)
    log_total = total.log()
    entropy = (log_total - (e * y).sum(1, keepdim=True) / total)[:, 0]
    out = []
    if tokens is not None:
        live = (tokens >= 0) & (tokens < x.shape[1])
        at = torch.where(live, tokens, torch.zeros_like(tokens))
        logp = y.gather(1, at) - log_total
        out.append(torch.where(live, logp, torch.zeros_like(logp)))
    out += [entropy, (m / tau + log_total)[:, 0]]
    if top:
        values, columns = _top(x, top)
        out += [(values - m) / tau - log_total, columns]
    out.append(torch.cat((m, log_total), 1))
    return tuple(out)


def _plain_logprobs_backward(s):
    x, tokens, tau = s["logits"], s["tokens"], s["case"]["temperature"]
    logq = (x.float() - s["stats"][:, :1]) / tau - s["stats"][:, 1:]
    pull = s["grad_lse"][:, None] - s["grad_entropy"][:, None] * (logq + s["entropy"][:, None])
    at, g = [], []
    if tokens is not None:
        live = (tokens >= 0) & (tokens < x.shape[1])
        at.append(torch.where(live, tokens, torch.zeros_like(tokens)))
        g.append(torch.where(live, s["grad_logprobs"], torch.zeros_like(s["grad_logprobs"])))
    if s["top_ids"] is not None:
        at.append(s["top_ids"])
        g.append(s["grad_top"])
    if at:
        at, g = torch.cat(at, 1), torch.cat(g, 1)
        pull = pull - g.sum(1, keepdim=True)
    grad = logq.exp() * pull
    if len(at):
        grad = grad.scatter_add(1, at, g)
    return (grad / tau).to(x.dtype)


def _plain_embed(s):
    ids, table = s["ids"], s["table"]
    live = (ids >= 0) & (ids < table.shape[0])
    rows = table[torch.where(live, ids, torch.zeros_like(ids))].float() * s["scale"]
    return torch.where(live[:, None], rows, torch.zeros_like(rows)).to(table.dtype)


def _plain_embed_grad(s):
    ids, vocab, width = s["ids"], s["case"]["vocab"], s["case"]["width"]
    live = (ids >= 0) & (ids < vocab)
    sums = torch.zeros(vocab + 1, width, device=ids.device)
    sums.index_add_(0, torch.where(live, ids, torch.full_like(ids, vocab)), s["grad"].float())
    return (sums[:vocab] * s["scale"]).to(_TYPES[s["case"]["out"]])


def _plain_embed_rows(s):
    """row_ids (ascending, -1 past the last), their rows, their number"""
    ids, vocab, width = s["ids"], s["case"]["vocab"], s["case"]["width"]
    n = s["rows"].shape[0]
    live = (ids >= 0) & (ids < vocab)
    named = torch.zeros(vocab + 1, dtype=torch.int64, device=ids.device)
    named.index_fill_(0, torch.where(live, ids, torch.full_like(ids, vocab)), 1)
    named[vocab] = 0
    place = named.cumsum(0)
    count = place[-1:].to(torch.int32)
    place = torch.where(named > 0, place - 1, torch.full_like(place, n))
    row_ids = torch.full((n + 1,), -1, dtype=torch.int64, device=ids.device)
    row_ids.index_copy_(0, place, torch.arange(vocab + 1, device=ids.device))
    row_ids[n] = -1
    sums = torch.zeros(n + 1, width, device=ids.device)
    sums.index_add_(0, place[torch.where(live, ids, torch.full_like(ids, vocab))], s["grad"].float())
    rows = (sums[:n] * s["scale"]).to(_TYPES[s["case"]["out"]])
    return row_ids[:n], rows, count


# ------------------------------------------------------- the least of work
def work(case):
    """Logits, grads and the table's named rows read once, outputs written
    once; the named rows of drawn tokens as many as are expected."""
    es = _BYTES[case["dtype"]]
    if case["op"] == "logprobs":
        rows, cols, k, top = case["rows"], case["cols"], case["k"], case["top"]
        if case["way"] == "fwd":
            return {"bytes": rows * (cols * es + k * 12 + 16 + top * 12), "flops": rows * cols * 6}
        return {"bytes": rows * (2 * cols * es + k * 12 + 20 + top * 12), "flops": rows * cols * 7}
    tokens, vocab, width, out = case["tokens"], case["vocab"], case["width"], _BYTES[case["out"]]
    live = tokens - case["masked"]
    named = int(-np.expm1(live * np.log1p(-_shares(vocab))).sum())
    if case["way"] == "fwd":
        return {"bytes": (named + tokens) * width * es + tokens * 8, "flops": tokens * width}
    read = live * width * es + tokens * 8
    if case["way"] == "grad":
        return {"bytes": read + vocab * width * out, "flops": live * width}
    return {"bytes": read + named * width * out + min(tokens, vocab) * 8, "flops": live * width}


# ------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """The same outputs from the definitions, in 64 bits."""
    s = prepare(case, seed)
    if case["op"] == "embed":
        return _exact_embed(case, s)
    rows, block = case["rows"], max(1, (1 << 25) // case["cols"])
    way = _exact_forward if case["way"] == "fwd" else _exact_backward
    parts = [way(case, s, slice(r, min(rows, r + block))) for r in range(0, rows, block)]
    if case["way"] == "bwd":
        return torch.cat(parts)
    return tuple(torch.cat(p) for p in zip(*parts))


def _exact_forward(case, s, at):
    x, tau, top = s["logits"][at].double(), case["temperature"], case["top"]
    logq = torch.log_softmax(x / tau, 1)
    out = []
    if s["tokens"] is not None:
        i = s["tokens"][at]
        gone = (i < 0) | (i >= case["cols"])
        out.append(logq.gather(1, i.clamp(0, case["cols"] - 1)).masked_fill(gone, 0))
    m = x.amax(1)
    out += [-(logq.exp() * logq).sum(1), torch.logsumexp(x / tau, 1)]
    if top:
        columns = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :top]
        out += [logq.gather(1, columns), columns]
    out.append(torch.stack((m, torch.logsumexp((x - m[:, None]) / tau, 1)), 1))
    return tuple(out)


def _exact_backward(case, s, at):
    x, tau, cols = s["logits"][at].double(), case["temperature"], case["cols"]
    z = (x / tau).requires_grad_(True)
    with torch.enable_grad():
        logq = torch.log_softmax(z, 1)
        lse = torch.logsumexp(z, 1)
        goal = (s["grad_lse"][at].double() * lse).sum()
        goal = goal - (s["grad_entropy"][at].double() * (logq.exp() * logq).sum(1)).sum()
        for ids, g in (("tokens", "grad_logprobs"), ("top_ids", "grad_top")):
            if s[ids] is None:
                continue
            i = s[ids][at]
            gone = (i < 0) | (i >= cols)
            picked = logq.gather(1, i.clamp(0, cols - 1)).masked_fill(gone, 0)
            goal = goal + (s[g][at].double() * picked).sum()
        grad, = torch.autograd.grad(goal, z)
    return grad / tau


def _exact_embed(case, s):
    ids, vocab, width = s["ids"], case["vocab"], case["width"]
    live = (ids >= 0) & (ids < vocab)
    if case["way"] == "fwd":
        out = torch.zeros(ids.shape[0], width, dtype=torch.float64, device=ids.device)
        out[live] = s["table"][ids[live]].double() * s["scale"]
        return out
    if case["way"] == "grad":
        sums = torch.zeros(vocab, width, dtype=torch.float64, device=ids.device)
        return sums.index_add_(0, ids[live], s["grad"][live].double()).mul_(s["scale"])
    names, place = torch.unique(ids[live], sorted=True, return_inverse=True)
    n, count = s["rows"].shape[0], names.shape[0]
    rows = torch.zeros(n, width, dtype=torch.float64, device=ids.device)
    rows.index_add_(0, place, s["grad"][live].double()).mul_(s["scale"])
    row_ids = torch.full((n,), -1, dtype=torch.int64, device=ids.device)
    row_ids[:count] = names
    return row_ids, rows, torch.tensor([count], dtype=torch.int32, device=ids.device)
