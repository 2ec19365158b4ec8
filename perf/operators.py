"""The language-model operators, as they are measured: their cases, their inputs, a pass through each.

Three operators, which a run of distillation from a teacher in 8 bits uses one after another:

* "logprob": the log probability of a given token for each row of logits, the entropy of the row and its top
  alternatives; for training, also the gradient of the first two;
* "distill": the divergence of a student's distribution from a teacher's top alternatives, with its gradient;
* "int8": a linear layer whose weight is held as 8-bit integers with a scale for each output channel, the input
  rounded to 8-bit integers with a scale for each token.

With `own` false, `run` computes them by elementary torch operations in 32 bits; with `own` true it calls the
package.  `exact` computes them in 64 bits from their definitions.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
IGNORE = -100                                    # a row without a given token


def listed():
    return [
        # one generated token of a Llama-3.1-8B-shaped model, with the 20 alternatives an answer's log shows
        dict(name="logprob_decode", op="logprob", rows=1, vocab=128256, type="bf16", top=20, temperature=1.0,
             masked=False, train="no"),
        # a batch of generated tokens of a GPT-2-shaped model (odd vocabulary), part of the vocabulary forbidden
        dict(name="logprob_serve", op="logprob", rows=64, vocab=50257, type="fp16", top=5, temperature=0.7,
             masked=True, train="no"),
        # a teacher's answers to a training batch: its 64 best tokens at each position
        dict(name="logprob_teacher", op="logprob", rows=2048, vocab=128256, type="bf16", top=64, temperature=2.0,
             masked=False, train="no"),
        # policy-gradient training: log probability and entropy, then the gradient of both
        dict(name="logprob_policy", op="logprob", rows=1023, vocab=50257, type="fp32", top=0, temperature=1.0,
             masked=False, train="entropy"),
        # next-token training of a Llama-2-13B-shaped model's head: log probability and gradient at once
        dict(name="logprob_nll", op="logprob", rows=4096, vocab=32000, type="bf16", top=0, temperature=1.0,
             masked=False, train="nll"),
        # a small distillation step in full precision, the teacher's 8 best tokens taken as the whole
        dict(name="distill_small", op="distill", rows=8, vocab=32000, type="fp32", top=8, temperature=1.0,
             masked=False, tail=False),
        # a GPT-2-shaped student, an odd number of rows, the rest of the vocabulary as one more outcome
        dict(name="distill_gpt2", op="distill", rows=501, vocab=50257, type="fp16", top=20, temperature=1.0,
             masked=True, tail=True),
        # a Llama-3.1-8B-shaped student at a training batch of 4096 tokens
        dict(name="distill_large", op="distill", rows=4096, vocab=128256, type="bf16", top=64, temperature=2.0,
             masked=False, tail=True),
        # one token through the widest layer of a Llama-3.1-8B-shaped model
        dict(name="int8_decode", op="int8", m=1, n=14336, k=4096, type="bf16", bias=False),
        # sixteen tokens through a GPT-2-shaped head (odd number of outputs)
        dict(name="int8_batch", op="int8", m=16, n=50257, k=768, type="fp16", bias=False),
        # a short prompt through a Llama-2-13B-shaped layer
        dict(name="int8_prompt", op="int8", m=200, n=13824, k=5120, type="bf16", bias=True),
        # a training batch through a Llama-3.1-8B-shaped layer
        dict(name="int8_large", op="int8", m=8192, n=14336, k=4096, type="bf16", bias=False),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("logprob", "distill", "int8"))
    kind = rng.choice(("bf16", "fp16", "fp32"))
    if op == "int8":
        while True:
            m, n, k = _spread(rng, 1, 8192), _spread(rng, 64, 60000), _spread(rng, 64, 14336)
            if m * n * k <= 8192 * 14336 * 4096 and m * n <= 8192 * 14336 and n * k <= 240 << 20:
                return dict(op=op, m=m, n=n, k=k, type=kind, bias=rng.random() < 0.5)
    most = (2048 if op == "logprob" else 4096) * 128256 // (2 if kind == "fp32" else 1)
    while True:
        rows, vocab = _spread(rng, 1, 4096), _spread(rng, 1000, 131072)
        if rows * vocab <= most:
            break
    case = dict(op=op, rows=rows, vocab=vocab, type=kind, temperature=rng.choice((1.0, 1.0, 0.7, 2.0)),
                masked=rng.random() < 0.3)
    if op == "logprob":
        case["train"] = rng.choice(("no", "no", "entropy", "nll"))
        case["top"] = 0 if case["train"] != "no" else rng.choice((0, 1, rng.randint(2, 64), 64))
    else:
        case["tail"] = rng.random() < 0.6
        case["top"] = _spread(rng, 1, 64)
    return case


def work(case):
    if case["op"] == "int8":
        m, n, k = case["m"], case["n"], case["k"]
        size = 4 if case["type"] == "fp32" else 2
        return {"bytes": size * m * k + n * k + 4 * n + size * m * n + (size * n if case["bias"] else 0),
                "flops": 2.0 * m * n * k}
    size = 4 if case["type"] == "fp32" else 2
    rows, vocab, top = case["rows"], case["vocab"], case["top"]
    both = case["op"] == "distill" or case["train"] != "no"
    # read the logits, write their gradient; the rows' own numbers and the alternatives
    return {"bytes": size * rows * vocab * (2 if both else 1) + rows * (20 + 12 * top),
            "flops": float(rows * vocab * (8 if both else 5))}


# ---- inputs -------------------------------------------------------------------------------------

def _logits(g, rows, vocab, kind, masked):
    """Logits of a language model: a skewed preference over the vocabulary, and each row's own part.  Where
    `masked`, tokens forbidden in the whole batch hold -inf, and some rows forbid half of the rest."""
    rank = torch.argsort(torch.rand(vocab, generator=g, device="cuda"))
    x = torch.randn(rows, vocab, generator=g, device="cuda").mul_(2.5).sub_(torch.log1p(rank.float()))
    x.add_(6.0)
    if masked:
        x[:, torch.rand(vocab, generator=g, device="cuda") < 0.3] = -math.inf
        some = torch.rand(rows, generator=g, device="cuda") < 0.25
        x.masked_fill_(some[:, None] & (torch.arange(vocab, device="cuda") % 2 == 1)[None], -math.inf)
        x[:, :64] = torch.randn(rows, 64, generator=g, device="cuda")          # always allowed
    return x.to(TYPES[kind])


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)
    if case["op"] == "int8":
        m, n, k, t = case["m"], case["n"], case["k"], TYPES[case["type"]]
        x = torch.randn(m, k, generator=g, device="cuda")
        x.mul_(torch.exp(0.5 * torch.randn(m, 1, generator=g, device="cuda")))     # tokens of unlike size
        x.mul_(1.0 + 9.0 * (torch.rand(k, generator=g, device="cuda") < 0.002))     # a few large channels
        codes = torch.randn(n, k, generator=g, device="cuda").mul_(32.0).round_().clamp_(-127, 127)
        scale = 0.02 * (0.5 + torch.rand(n, generator=g, device="cuda")) / 32.0
        bias = 0.1 * torch.randn(n, generator=g, device="cuda") if case["bias"] else None
        return dict(x=x.to(t), codes=codes.to(torch.int8), scale=scale, bias=None if bias is None else bias.to(t))
    rows, vocab, top = case["rows"], case["vocab"], case["top"]
    data = dict(logits=_logits(g, rows, vocab, case["type"], case["masked"]))
    unit = 4096.0 if case["type"] == "fp16" else 1.0          # training in fp16 scales its loss
    if case["op"] == "logprob":
        # given tokens are ones that the row can give: among the best of a few tries
        tries = torch.randint(0, vocab, (rows, 8), generator=g, device="cuda")
        tries[:, 0] %= min(64, vocab)
        best = data["logits"].gather(1, tries).float().argmax(1, keepdim=True)
        target = tries.gather(1, best).squeeze(1)
        if rows > 8:                                   # prompt positions carry no given token
            target[torch.rand(rows, generator=g, device="cuda") < 0.1] = IGNORE
        data["targets"] = target
        if case["train"] == "entropy":
            data["grad_logprob"] = torch.randn(rows, generator=g, device="cuda") * (unit / rows)
            data["grad_entropy"] = torch.full((rows,), -0.01 * unit / rows, device="cuda")
        elif case["train"] == "nll":
            data["grad_logprob"] = torch.full((rows,), -unit / rows, device="cuda")
        return data
    # a teacher near the student: its best tokens and their log probabilities at the same temperature
    ids, logp = [], []
    for r in range(0, rows, 512):
        z = data["logits"][r:r + 512].float()
        z = (z + torch.randn(z.shape, generator=g, device="cuda")) / case["temperature"]
        v, i = torch.topk(z, top, dim=1)
        ids.append(i)
        logp.append(v - torch.logsumexp(z, 1, keepdim=True))
    data["top_id"], data["top_logprob"] = torch.cat(ids), torch.cat(logp)
    data["grad_loss"] = torch.rand(rows, generator=g, device="cuda") * (unit / rows)
    return data


def prepare(case, seed):
    state = _inputs(case, seed)
    state["case"] = case
    if own and case["op"] == "int8":
        from compressed_adamw_state_amd import int8
        state["weight"] = int8.Int8Weight.from_codes(state["codes"], state["scale"])
    if case["op"] == "logprob" and case["train"] == "entropy":
        state["logits"].requires_grad_(own)
    return state


# ---- one pass -----------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"logprob": _own_logprob, "distill": _own_distill, "int8": _own_int8}[op](state)
    return {"logprob": _plain_logprob, "distill": _plain_distill, "int8": _plain_int8}[op](state)


def _own_logprob(s):
    from compressed_adamw_state_amd import losses
    c = s["case"]
    if c["train"] == "nll":
        r = losses.token_logprobs_grad(s["logits"], s["targets"], s["grad_logprob"], temperature=c["temperature"])
        return {"logprob": r.logprob, "entropy": r.entropy, "grad": r.grad}
    r = losses.token_logprobs(s["logits"], s["targets"], top=c["top"], temperature=c["temperature"])
    if c["train"] == "entropy":
        grad, = torch.autograd.grad((r.logprob, r.entropy), s["logits"], (s["grad_logprob"], s["grad_entropy"]))
        return {"logprob": r.logprob.detach(), "entropy": r.entropy.detach(), "grad": grad}
    out = {"logprob": r.logprob, "entropy": r.entropy}
    if c["top"]:
        out.update(top_logprob=r.top_logprob, top_id=r.top_id)
    return out


def _own_distill(s):
    from compressed_adamw_state_amd import losses
    c = s["case"]
    loss, grad = losses.distill_grad(s["logits"], s["top_id"], s["top_logprob"], s["grad_loss"],
                                     temperature=c["temperature"], tail=c["tail"])
    return {"loss": loss, "grad": grad}


def _own_int8(s):
    from compressed_adamw_state_amd import int8
    return int8.int8_linear(s["x"], s["weight"], s["bias"])


def _plain_logprob(s):
    c, x, target = s["case"], s["logits"], s["targets"]
    z = x.float() * (1.0 / c["temperature"])
    d = z - z.amax(1, keepdim=True)
    e = torch.exp(d)
    total = e.sum(1, keepdim=True)
    logs = d - torch.log(total)
    given = (target >= 0) & (target < c["vocab"])
    at = torch.where(given, target, 0)
    logprob = torch.where(given, logs.gather(1, at[:, None]).squeeze(1), 0.0)
    p = e / total
    entropy = -torch.where(p > 0, p * logs, 0.0).sum(1)
    out = {"logprob": logprob, "entropy": entropy}
    if c["top"]:
        order = torch.sort(x, dim=1, descending=True, stable=True)[1][:, :c["top"]]
        out.update(top_logprob=logs.gather(1, order), top_id=order)
    if c["train"] != "no":
        g = torch.where(given, s["grad_logprob"], 0.0)
        grad = -g[:, None] * p
        if c["train"] == "entropy":
            grad = grad - torch.where(p > 0, s["grad_entropy"][:, None] * p * (logs + entropy[:, None]), 0.0)
        grad.scatter_add_(1, at[:, None], g[:, None])
        out["grad"] = (grad * (1.0 / c["temperature"])).to(x.dtype)
    return out


def _plain_distill(s):
    c, x, ids, t = s["case"], s["logits"], s["top_id"], s["top_logprob"]
    z = x.float() * (1.0 / c["temperature"])
    d = z - z.amax(1, keepdim=True)
    e = torch.exp(d)
    total = e.sum(1, keepdim=True)
    logs = d - torch.log(total)
    p = e / total
    q = torch.exp(t)
    if not c["tail"]:
        q = q / q.sum(1, keepdim=True)
    logq = torch.log(q)
    loss = torch.where(q > 0, q * (logq - logs.gather(1, ids)), 0.0).sum(1)
    grad = p * (s["grad_loss"] * (1.0 / c["temperature"]))[:, None]
    if c["tail"]:
        rest = p.scatter(1, ids, 0.0)                             # the vocabulary outside the alternatives
        left = rest.sum(1, keepdim=True)
        q_left = (1.0 - q.sum(1, keepdim=True)).clamp_min(0.0)
        here = (q_left > 0) & (left > 0)
        loss = loss + torch.where(here, q_left * (torch.log(q_left) - torch.log(left)), 0.0).squeeze(1)
        share = torch.where(here, q_left / left, 0.0)
        grad = grad - rest * (share * (s["grad_loss"] * (1.0 / c["temperature"]))[:, None])
    grad.scatter_add_(1, ids, -q * (s["grad_loss"] * (1.0 / c["temperature"]))[:, None])
    return {"loss": loss, "grad": grad.to(x.dtype)}


def _plain_int8(s):
    x = s["x"]
    # 16-bit inputs: 127 x is exact in 32 bits and the quotient of two such numbers is never rounded onto a
    # border between two codes; 32-bit inputs next to a border need 64
    w = x.double() if x.dtype == torch.float32 else x.float()
    most = w.abs().amax(1, keepdim=True)
    codes = torch.where(most > 0, torch.round(w * 127.0 / most), 0.0).float()
    scale = (most / 127.0).float()
    y = (codes @ s["codes"].float().t()) * (scale * s["scale"])
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(x.dtype)


# ---- the definitions in 64 bits -----------------------------------------------------------------

def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "int8":
        x = s["x"].to(torch.float64)
        peak = x.abs().max(dim=1).values
        q = torch.round(127.0 * x / torch.where(peak > 0, peak, 1.0)[:, None])
        out = []
        w = s["codes"].to(torch.float64).t().contiguous()
        for r in range(0, case["m"], 1024):
            y = torch.mm(q[r:r + 1024], w) * (peak[r:r + 1024] / 127.0)[:, None] * s["scale"].double()[None]
            out.append(y if s["bias"] is None else y + s["bias"].double()[None])
        return torch.cat(out)
    parts = [(_exact_logprob if case["op"] == "logprob" else _exact_distill)(case, s, r, min(r + 256, case["rows"]))
             for r in range(0, case["rows"], 256)]
    return {k: torch.cat([p[k] for p in parts]) for k in parts[0]}


def _exact_logprob(case, s, a, b):
    x = s["logits"][a:b]
    z = x.double() / case["temperature"]
    lse = torch.logsumexp(z, 1)
    prob = torch.exp(z - lse[:, None])
    target = s["targets"][a:b]
    rows = torch.arange(b - a, device=x.device)
    has = target != IGNORE
    lp = torch.zeros(b - a, dtype=torch.float64, device=x.device)
    lp[has] = z[rows[has], target[has]] - lse[has]
    ent = torch.special.entr(prob).sum(1)
    out = {"logprob": lp, "entropy": ent}
    if case["top"]:
        # one whole number for each entry: its rank among the values, then its place from the end
        bits = (x.float() + 0.0).view(torch.int32).long()
        key = torch.where(bits < 0, -(bits & 0x7FFFFFFF) - 1, bits)
        key = key * (1 << 20) + ((1 << 20) - 1 - torch.arange(case["vocab"], device=x.device))
        order = torch.topk(key, case["top"], dim=1).indices
        out.update(top_logprob=z.gather(1, order) - lse[:, None], top_id=order)
    if case["train"] != "no":
        gl = torch.where(has, s["grad_logprob"][a:b].double(), 0.0)
        grad = -prob * gl[:, None]
        grad[rows[has], target[has]] += gl[has]
        if case["train"] == "entropy":
            # dH/dz_j = entr(p_j) - p_j H
            grad += s["grad_entropy"][a:b].double()[:, None] * (torch.special.entr(prob) - prob * ent[:, None])
        out["grad"] = grad / case["temperature"]
    return out


def _exact_distill(case, s, a, b):
    x, ids = s["logits"][a:b], s["top_id"][a:b]
    z = x.double() / case["temperature"]
    lse = torch.logsumexp(z, 1, keepdim=True)
    q = torch.exp(s["top_logprob"][a:b].double())
    if not case["tail"]:
        q = q / q.sum(1, keepdim=True)
    loss = torch.special.xlogy(q, q).sum(1) - (q * (z.gather(1, ids) - lse)).sum(1)
    # the target's distribution over the vocabulary: the rest of it is shared out as the student shares it
    goal = torch.zeros_like(z)
    if case["tail"]:
        outside = z.scatter(1, ids, -math.inf)
        rest = torch.logsumexp(outside, 1, keepdim=True)
        more = torch.clamp(1.0 - q.sum(1, keepdim=True), min=0.0)
        use = (more > 0) & (rest > -math.inf)
        more = torch.where(use, more, 0.0)
        loss = loss + (torch.special.xlogy(more, more) - torch.where(use, more * (rest - lse), 0.0)).squeeze(1)
        goal = torch.where(use, more * torch.exp(outside - rest), 0.0)
    goal.scatter_(1, ids, q)
    grad = (torch.exp(z - lse) - goal) * s["grad_loss"][a:b].double()[:, None] / case["temperature"]
    return {"loss": loss, "grad": grad}
