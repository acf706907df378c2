"""Cases and plain forms of the operators on the logits of a verification pass.

A pass leaves one row of target logits per mask slot; ``ssv.accept`` decides on them.  What a server
returns beside the tokens, and what trains a drafter on the target's answers, comes from the same rows:

* ``logprobs``  ssv.logprobs: of each entry's row and token, the log-probability, the token's rank, the
                row's entropy and log-sum-exp, and its top alternatives;
* ``distill``   ssv.distill: loss of a drafter's logits against the target's top alternatives (as
                ssv.logprobs writes them), alone or with its gradient;
* ``backward``  ssv.distill_backward: the gradient for given upstream gradients of the row losses.

Plain forms are elementary torch operations in 32 bits; ``exact`` restates each operator in 64 bits.
"""
import math
import random

import torch

own = False

VOCAB = 151936


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
# n: entries; vocab; pad: elements between the end of a row and the next; dtype of the logits; k: top alternatives;
# temp: temperature; idle: percent of entries without a token (or of rows of weight 0)
def listed():
    return [
        # one emitted token of one request, twenty alternatives: a chat server's smallest call
        dict(name="logprobs 1 row", op="logprobs", n=1, vocab=VOCAB, pad=0, dtype="bf16", k=20, temp=1.0, idle=0, masked=0, picked=False),
        # one pass of the 8-sequence decode workload, blocks of 8
        dict(name="logprobs decode 64", op="logprobs", n=64, vocab=VOCAB, pad=0, dtype="bf16", k=20, temp=1.0, idle=0, masked=0, picked=True),
        # the mixed decode batch: 64 sequences with blocks of 4..32, fp32 logits, rejected stages without a token, the 32
        # alternatives that an order predictor reads
        dict(name="logprobs mixed 960 fp32", op="logprobs", n=960, vocab=VOCAB, pad=0, dtype="f32", k=32, temp=1.5, idle=30, masked=0, picked=True),
        # a prompt of 8192 tokens scored, no alternatives
        dict(name="logprobs prompt 8192", op="logprobs", n=8192, vocab=VOCAB, pad=0, dtype="bf16", k=0, temp=1.0, idle=0, masked=0, picked=False),
        # a small vocabulary of odd size under a grammar's mask, rows cut out of a wider buffer
        dict(name="logprobs grammar 300", op="logprobs", n=300, vocab=9001, pad=6, dtype="f32", k=64, temp=0.7, idle=5, masked=90, picked=True),
        # the loss alone, on the slots of one request: what a drafter is watched by
        dict(name="distill loss 32", op="distill", n=32, vocab=VOCAB, pad=0, dtype="bf16", k=32, temp=1.0, idle=0, rest=True, grad=False),
        # a training step's loss and gradient: 64 blocks of 16 with the position weights of block drafting
        dict(name="distill 1024", op="distill", n=1024, vocab=VOCAB, pad=0, dtype="bf16", k=64, temp=1.0, idle=10, rest=False, grad=True),
        # a large step with as many alternatives as are kept
        dict(name="distill 4096", op="distill", n=4096, vocab=VOCAB, pad=0, dtype="bf16", k=128, temp=2.0, idle=0, rest=True, grad=True),
        # fp32 logits over a small odd vocabulary
        dict(name="distill odd fp32", op="distill", n=700, vocab=32003, pad=0, dtype="f32", k=50, temp=1.0, idle=20, rest=True, grad=True),
        # the gradient alone, on one request's slots
        dict(name="backward 32", op="backward", n=32, vocab=VOCAB, pad=0, dtype="bf16", k=20, temp=1.0, idle=0, rest=True),
        # fp32 logits of a large step
        dict(name="backward 1500 fp32", op="backward", n=1500, vocab=VOCAB, pad=0, dtype="f32", k=64, temp=1.0, idle=10, rest=True),
        # an odd vocabulary with padded rows
        dict(name="backward odd", op="backward", n=2000, vocab=9001, pad=7, dtype="bf16", k=32, temp=1.5, idle=10, rest=False),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["logprobs", "logprobs", "distill", "backward"])
    vocab = rng.choice([256, VOCAB, VOCAB, spread(200, 200000), spread(200, 200000) | 1])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    n = spread(1, min(8000, 1200000000 // (vocab * (4 if dtype == "f32" else 2))))
    c = dict(op=op, n=n, vocab=vocab, pad=rng.choice([0, 0, 0, 1, 8, 64]), dtype=dtype,
             temp=rng.choice([1.0, 1.0, 0.7, 1.5, 2.0]), idle=rng.choice([0, 0, 10, 40]))
    if op == "logprobs":
        return c | dict(k=rng.choice([0, 1, 5, 20, 32, 64, 128]), masked=rng.choice([0, 0, 0, 50, 95]), picked=rng.random() < 0.5)
    c |= dict(k=rng.choice([1, 8, 20, 32, 50, 64, 100, 128]), rest=rng.random() < 0.5)
    return c | dict(grad=rng.random() < 0.75) if op == "distill" else c


def _idle(case):
    """Entries without a token, rows of weight 0: shapes do not follow the seed."""
    r = random.Random(case["n"] * 1000 + case["idle"])
    return [r.random() * 100 < case["idle"] for _ in range(case["n"])]


def work(case):
    n = case["n"]
    live = n - sum(_idle(case))
    es = 4 if case["dtype"] == "f32" else 2
    row, k = case["vocab"] * es, case["k"]
    if case["op"] == "logprobs":
        return dict(bytes=float(live * row + n * (8 + 16 + 8 * k)), flops=float(live * case["vocab"] * 8))
    teacher = n * (8 * k + 4)
    if case["op"] == "backward":
        return dict(bytes=float(live * row + n * row + teacher + 12 * n), flops=float(live * case["vocab"] * 5))
    return dict(bytes=float(live * row + (n * row if case["grad"] else 0) + teacher + 12 * n),
                flops=float(live * case["vocab"] * (10 if case["grad"] else 5)))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _rows(g, rows, case, dt):
    """Logits of a language model: a wide bulk and forty tokens that stand out.  Returns the rows (of a buffer `pad`
    elements wider) and those tokens."""
    v = case["vocab"]
    buf = torch.empty(rows, v + case["pad"], dtype=dt, device="cuda")
    x = buf[:, :v]
    peaks = torch.randint(0, v, (rows, 40), generator=g, device="cuda")
    up = 6.0 + torch.empty(rows, 40, device="cuda").exponential_(0.4, generator=g).clamp_(max=12)
    step = max(1, (1 << 29) // v)
    for i in range(0, rows, step):
        y = torch.randn(min(step, rows - i), v, generator=g, device="cuda").mul_(2.0)
        x[i:i + step] = y.scatter_add_(1, peaks[i:i + step], up[i:i + step]).to(dt)
    if case["pad"]:
        buf[:, v:] = 1e4
    return x, peaks


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    n, v, k = case["n"], case["vocab"], case["k"]
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    idle = torch.tensor(_idle(case), device="cuda")
    s = dict(op=case["op"], temp=case["temp"], k=k)
    if case["op"] == "logprobs":
        x, peaks = _rows(g, n, case, dt)
        rows = None
        if case["picked"]:      # entries in the order of the stages, rows in the order of the slots
            rows = torch.randperm(n, generator=g, device="cuda")
        at = peaks if rows is None else peaks[rows]
        tok = at.gather(1, torch.randint(0, 40, (n, 1), generator=g, device="cuda"))[:, 0]
        if case["masked"]:
            step = max(1, (1 << 29) // v)
            for i in range(0, n, step):
                out = torch.rand(min(step, n - i), v, generator=g, device="cuda") * 100 < case["masked"]
                out.scatter_(1, peaks[i:i + step], False)
                x[i:i + step].masked_fill_(out, float("-inf"))
        s |= dict(logits=x, tokens=torch.where(idle, -1, tok).int(), rows=None if rows is None else rows.int())
        return s
    z, _ = _rows(g, n, case, dt)
    token = torch.empty(n, k, dtype=torch.int32, device="cuda")
    logp = torch.empty(n, k, device="cuda")
    step = max(1, (1 << 28) // v)
    for i in range(0, n, step):     # the target's rows: near the drafter's, read through their top k
        t = torch.randn(min(step, n - i), v, generator=g, device="cuda").add_(z[i:i + step]).div_(case["temp"])
        top, at = t.topk(k, 1)
        logp[i:i + step] = top - torch.logsumexp(t, 1, keepdim=True)
        token[i:i + step] = at.int()
    some = torch.rand(n, generator=g, device="cuda") < 0.1          # rows with fewer alternatives
    cut = (torch.arange(k, device="cuda") >= (k + 1) // 2)[None] & some[:, None]
    token.masked_fill_(cut, -1)
    logp.masked_fill_(cut, float("-inf"))
    stage = torch.arange(n, device="cuda") % 16
    w = torch.exp(-stage.float() / 7.0) / max(1, n)
    s |= dict(logits=z, token=token, logp=logp, weight=torch.where(idle, 0.0, w), rest=case["rest"])
    if case["op"] == "distill":
        return s | dict(grad=case["grad"])
    # a training step keeps the statistics of its forward pass: maximum and sum, relative to it, of exp(z / T), over the
    # row and over the tokens that are not the target's
    stats = torch.empty(n, 4, device="cuda")
    for i in range(0, n, step):
        y = z[i:i + step].double()
        for j in (0, 2):
            m = y.amax(1)
            stats[i:i + step, j] = m.float()
            stats[i:i + step, j + 1] = ((y - m[:, None]) / case["temp"]).exp().sum(1).float()
            own_rows, c = (token[i:i + step] >= 0).nonzero(as_tuple=True)
            y[own_rows, token[i:i + step][own_rows, c].long()] = float("-inf")
    return s | dict(stats=stats, grad_loss=torch.randn(n, generator=g, device="cuda"))


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    op = s["op"]
    if own:
        from diffusion_speculative_verification_gb300 import ssv
        if op == "logprobs":
            logprob, rank, entropy, lse, top_logprob, top_token = ssv.logprobs(
                s["logits"], s["tokens"], top_k=s["k"], T=s["temp"], rows=s["rows"])
            out = dict(logprob=logprob, rank=rank, entropy=entropy, lse=lse)
            return out | dict(top_logprob=top_logprob, top_token=top_token) if s["k"] else out
        mode = ssv.REST if s["rest"] else ssv.RENORM
        if op == "distill":
            loss, stats, grad = ssv.distill(s["logits"], s["token"], s["logp"], T=s["temp"], mode=mode, weight=s["weight"],
                                            grad=s["grad"])
            return dict(loss=loss, grad=grad) if s["grad"] else dict(loss=loss)
        return dict(grad=ssv.distill_backward(s["logits"], s["token"], s["logp"], s["stats"], s["grad_loss"], T=s["temp"],
                                              mode=mode, weight=s["weight"]))
    return dict(logprobs=_logprobs, distill=_distill, backward=_backward)[op](s)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _chunks(n, v):
    step = max(1, (1 << 28) // v)
    return [slice(i, min(n, i + step)) for i in range(0, n, step)]


def _logprobs(s):
    tokens, k = s["tokens"].long(), s["k"]
    n, v = len(tokens), s["logits"].shape[1]
    dev = tokens.device
    live = tokens >= 0
    out = dict(logprob=torch.empty(n, device=dev), rank=torch.empty(n, dtype=torch.int32, device=dev),
               entropy=torch.empty(n, device=dev), lse=torch.empty(n, device=dev))
    if k:
        out |= dict(top_logprob=torch.empty(n, k, device=dev), top_token=torch.empty(n, k, dtype=torch.int32, device=dev))
    col = torch.arange(v, device=dev)
    for c in _chunks(n, v):
        x = (s["logits"][c] if s["rows"] is None else s["logits"][s["rows"][c].long()]).float()
        t = tokens[c].clamp(min=0)[:, None]
        m = x.amax(1, keepdim=True)
        y = (x - m) / s["temp"]
        e = y.exp()
        total = e.sum(1, keepdim=True)
        log = total.log()
        mean = torch.where(e > 0, e * y, 0.0).sum(1, keepdim=True) / total
        own_x = x.gather(1, t)
        before = ((x > own_x) | ((x == own_x) & (col < t))).sum(1)
        out["logprob"][c] = torch.where(live[c], (y.gather(1, t) - log)[:, 0], 0.0)
        out["rank"][c] = torch.where(live[c], before + 1, 0).int()
        out["entropy"][c] = torch.where(live[c], (log - mean)[:, 0], 0.0)
        out["lse"][c] = torch.where(live[c], (m / s["temp"] + log)[:, 0], 0.0)
        if not k:
            continue
        # value and column in one ordered number: ties go to the lowest column
        b = (x + 0.0).view(torch.int32).long()
        b = torch.where(b < 0, -(b & 0x7FFFFFFF), b)
        at = (((b << 24) | (v - 1 - col)).topk(min(k, v), 1).values & 0xFFFFFF).neg_().add_(v - 1)
        val = x.gather(1, at)
        lp, at = (val - m) / s["temp"] - log, at.int()
        none = (val == float("-inf")) | ~live[c][:, None]
        out["top_logprob"][c] = torch.nn.functional.pad(lp.masked_fill(none, float("-inf")), (0, k - at.shape[1]), value=float("-inf"))
        out["top_token"][c] = torch.nn.functional.pad(at.masked_fill(none, -1), (0, k - at.shape[1]), value=-1)
    return out


def _target(s, c):
    """Of the rows c: the target's probabilities and their logarithms, what they leave to the rest, their sum with it (64
    bits: the rest is a small difference); absent entries have 0."""
    there = s["token"][c] >= 0
    t = torch.where(there, s["logp"][c], float("-inf")).double()
    if s["rest"]:
        p = t.exp()
        r = (1.0 - p.sum(1, keepdim=True)).clamp(min=0.0)
    else:
        p = (t - t.amax(1, keepdim=True)).exp()
        p = p / p.sum(1, keepdim=True)
        t = p.log()
        r = torch.zeros_like(p[:, :1])
    return there, p, t, r, p.sum(1, keepdim=True) + r


def _others(y, there, token):
    """The rows without the target's tokens."""
    own_rows, c = there.nonzero(as_tuple=True)
    y = y.clone()
    y[own_rows, token[own_rows, c]] = float("-inf")
    return y


def _gradient(x, there, token, p, r, total, sums, factor, temp):
    """factor / temp * (total q - p) at the target's tokens; their own softmax times (total u - r) at the others."""
    p, r, total = p.float(), r.float(), total.float()
    m, s, mr, sr = sums
    u = (((mr - m) / temp).double().exp() * sr / s).float()
    grad = ((x - mr) / temp).exp() * ((total * u - r) / sr)
    at_top = total * (((x.gather(1, token) - m) / temp).exp() / s) - p
    own_rows, c = there.nonzero(as_tuple=True)
    grad[own_rows, token[own_rows, c]] = at_top[own_rows, c]
    return grad * (factor[:, None] / temp)


def _distill(s):
    n, v = s["logits"].shape
    out = dict(loss=torch.empty(n, device=s["weight"].device))
    if s["grad"]:
        out["grad"] = torch.empty(n, v, dtype=s["logits"].dtype, device=s["weight"].device)
    for c in _chunks(n, v):
        x = s["logits"][c].float()
        there, p, t, r, total = _target(s, c)
        token = s["token"][c].long().clamp(min=0)
        w = s["weight"][c]
        # a loss is a small difference of logarithms: those, a few per row, in 64 bits; the sums over the row in 32
        m = x.amax(1, keepdim=True)
        z = _others(x, there, token)
        mr = z.amax(1, keepdim=True)
        total_e = ((x - m) / s["temp"]).exp().sum(1, keepdim=True)
        rest_e = ((z - mr) / s["temp"]).exp().sum(1, keepdim=True)
        log = total_e.double().log()
        loss = torch.where(p > 0, p * (t - ((x.gather(1, token) - m).double() / s["temp"] - log)), 0.0).sum(1)
        log_u = (mr - m).double() / s["temp"] + rest_e.double().log() - log
        rest = torch.where(r > 0, r * (r.log() - log_u), 0.0)[:, 0]
        out["loss"][c] = torch.where(w != 0, w * (loss + rest), 0.0).float()
        if s["grad"]:
            grad = _gradient(x, there, token, p, r, total, (m, total_e, mr, rest_e), w, s["temp"])
            out["grad"][c] = torch.where((w != 0)[:, None], grad, 0.0).to(s["logits"].dtype)
    return out


def _backward(s):
    n, v = s["logits"].shape
    grad = torch.empty(n, v, dtype=s["logits"].dtype, device=s["weight"].device)
    for c in _chunks(n, v):
        there, p, _, r, total = _target(s, c)
        w = s["weight"][c]
        x = _gradient(s["logits"][c].float(), there, s["token"][c].long().clamp(min=0), p, r, total,
                      s["stats"][c].split(1, 1), w * s["grad_loss"][c], s["temp"])
        grad[c] = torch.where((w != 0)[:, None], x, 0.0).to(grad.dtype)
    return dict(grad=grad)


# ---------------------------------------------------------------------------
# 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    n, v = s["logits"].shape
    f64 = torch.float64
    step = max(1, (1 << 27) // v)
    if case["op"] == "logprobs":
        k = s["k"]
        out = {name: torch.zeros(n, dtype=f64, device="cuda") for name in ("logprob", "entropy", "lse")} | dict(rank=None)
        if k:
            out |= dict(top_logprob=torch.full((n, k), -math.inf, dtype=f64, device="cuda"), top_token=None)
        where = torch.arange(n, device="cuda") if s["rows"] is None else s["rows"].long()
        live = (s["tokens"] >= 0).nonzero()[:, 0]
        for i in range(0, len(live), step):
            e = live[i:i + step]
            lp = s["logits"][where[e]].double() / s["temp"]
            lse = torch.logsumexp(lp, 1)
            lp = lp - lse[:, None]
            out["lse"][e] = lse
            out["logprob"][e] = lp[torch.arange(len(e), device="cuda"), s["tokens"][e].long()]
            out["entropy"][e] = -torch.nan_to_num(lp.exp() * lp, nan=0.0).sum(1)
            if k:
                top = torch.topk(lp, min(k, v), 1).values
                out["top_logprob"][e, :top.shape[1]] = top
        return out
    scale = s["weight"].double()
    if case["op"] == "backward":
        scale = scale * s["grad_loss"].double()
    loss = torch.zeros(n, dtype=f64, device="cuda")
    grad = torch.zeros(n, v, dtype=f64, device="cuda") if case.get("grad", True) else None
    live = (s["weight"] != 0).nonzero()[:, 0]
    for i in range(0, len(live), step):
        e = live[i:i + step]
        logq = torch.log_softmax(s["logits"][e].double() / s["temp"], 1)
        t, at = s["logp"][e].double(), s["token"][e].long()
        if not s["rest"]:
            t = torch.log_softmax(t, 1)
        p = torch.zeros_like(logq).scatter_add_(1, at.clamp(min=0), torch.where(at >= 0, t.exp(), 0.0))
        listed_ = torch.zeros_like(logq).scatter_add_(1, at.clamp(min=0), (at >= 0).double()) > 0
        mass = p.sum(1)
        r = (1 - mass).clamp(min=0) if s["rest"] else torch.zeros_like(mass)
        log_u = torch.logsumexp(logq.masked_fill(listed_, -math.inf), 1)
        cross = torch.xlogy(p, p) - torch.where(listed_ & (p > 0), p * logq, 0.0)
        loss[e] = s["weight"][e].double() * (cross.sum(1) + torch.xlogy(r, r) - torch.where(r > 0, r * log_u, 0.0))
        if grad is not None:
            # the rest's share r spread over the tokens that are not listed as the drafter spreads its own
            p += torch.where(listed_, 0.0, (logq - log_u[:, None]).exp() * r[:, None])
            grad[e] = ((mass + r)[:, None] * logq.exp() - p) * (scale[e, None] / s["temp"])
    if case["op"] == "backward":
        return dict(grad=grad)
    return dict(loss=loss) if grad is None else dict(loss=loss, grad=grad)
