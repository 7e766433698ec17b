"""Measured cases of the operators that work on whole rows of vocabulary logits.

sample    a token per row of logits [R, V] with temperature, top-k, top-p and min-p, from given
          uniform numbers: the target model's answers, and the anchors that a draft block starts
          from.
distill   the loss that trains a drafter on its target's top logits (the ids and scores that the
          top-k pass keeps), its gradient, and both in one call.

A case is a plain dict; `run` computes it in elementary torch operations, or, where `own` is
true, through the package's entry points.
"""
import math

import torch

own = False

DEVICE = "cuda"

# Vocabularies and row counts are those of the selector's workloads (a draft block of 16
# positions; 64 sequences, 32 sequences of the larger vocabulary) and generic odd ones.


def listed():
    return [
        # one sequence decoding with a nucleus: the whole call is latency
        dict(name="sample-one-row", op="sample", rows=1, vocab=151936, dtype="bf16",
             params="top_p"),
        # a serving batch, every request with settings of its own (greedy ones among them)
        dict(name="sample-batch-64", op="sample", rows=64, vocab=151936, dtype="bf16",
             params="mixed"),
        # the target's answers at every position of 64 draft blocks
        dict(name="sample-blocks-1024", op="sample", rows=1024, vocab=151936, dtype="bf16",
             params="mixed"),
        # the larger vocabulary with one top-k and top-p for all rows
        dict(name="sample-top-k-512", op="sample", rows=512, vocab=262144, dtype="bf16",
             params="top_k_top_p"),
        # float32 logits, a vocabulary whose rows are not aligned, no truncation
        dict(name="sample-f32-odd", op="sample", rows=37, vocab=50021, dtype="f32",
             params="plain"),
        # float32 logits of many rows, settings mixed
        dict(name="sample-f32-256", op="sample", rows=256, vocab=151936, dtype="f32",
             params="mixed"),
        # the loss of one draft block, as an evaluation asks for it
        dict(name="distill-loss-block", op="distill", rows=16, vocab=151936, k=16, dtype="bf16",
             temperature=1.0, direction="forward"),
        # the loss alone for 64 draft blocks, softened
        dict(name="distill-loss-1024", op="distill", rows=1024, vocab=151936, k=64, dtype="bf16",
             temperature=2.0, direction="forward"),
        # the gradient from kept row statistics, larger vocabulary
        dict(name="distill-gradient-512", op="distill", rows=512, vocab=262144, k=32,
             dtype="bf16", temperature=1.0, direction="backward"),
        # float32 logits, rows that are not aligned: loss and gradient
        dict(name="distill-step-f32-odd", op="distill", rows=131, vocab=32003, k=7, dtype="f32",
             temperature=1.5, direction="step"),
        # a training step on 64 draft blocks
        dict(name="distill-step-1024", op="distill", rows=1024, vocab=151936, k=16, dtype="bf16",
             temperature=1.0, direction="step"),
        # a large training step: 256 draft blocks
        dict(name="distill-step-4096", op="distill", rows=4096, vocab=151936, k=32, dtype="bf16",
             temperature=1.0, direction="step"),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    vocab = _log_uniform(rng, 1000, 262144)
    if rng.random() < 0.5:
        vocab |= 1
    dtype = rng.choice(["bf16", "bf16", "f32"])
    # no more than the largest listed case: rows times bytes of a row
    most = min(1500, 300_000_000 // (vocab * (2 if dtype == "bf16" else 4)))
    rows = _log_uniform(rng, 1, most)
    if rng.random() < 0.5:
        return dict(op="sample", rows=rows, vocab=vocab, dtype=dtype,
                    params=rng.choice(["mixed", "top_p", "top_k_top_p", "min_p", "plain"]))
    return dict(op="distill", rows=rows, vocab=vocab, k=_log_uniform(rng, 1, 64), dtype=dtype,
                temperature=rng.choice([0.75, 1.0, 1.5, 2.0, 4.0]),
                direction=rng.choice(["forward", "backward", "step", "step"]))


# ---- inputs ------------------------------------------------------------------------------------

def _torch_dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device=DEVICE)


def _distinct_ids(g, rows, vocab, k):
    """k distinct ids per row: one from each of k equal parts of the vocabulary."""
    part = vocab // k
    ids = torch.arange(k, device=DEVICE) * part + (_rand(g, rows, k) * part).long()
    return ids


def _logits(g, case):
    """Normal logits with a few raised tokens in each row, and one that stands out in half of the
    rows: the rows where a model hesitates and those where it is sure."""
    rows, vocab = case["rows"], case["vocab"]
    x = torch.randn(rows, vocab, generator=g, device=DEVICE) * 2.5
    raised = _distinct_ids(g, rows, vocab, 8)
    x.scatter_add_(1, raised, 4.0 + 6.0 * _rand(g, rows, 8))
    sure = torch.where(_rand(g, rows, 1) < 0.5, 8.0, 0.0)
    x.scatter_add_(1, raised[:, :1], sure)
    return x


def _pick(g, rows, values, dtype=torch.float32):
    t = torch.tensor(values, device=DEVICE, dtype=dtype)
    return t[(_rand(g, rows) * len(values)).long()]


def prepare(case, seed):
    g = _generator(seed)
    rows = case["rows"]
    if case["op"] == "sample":
        logits = _logits(g, case).to(_torch_dtype(case))
        uniforms = _rand(g, rows)
        p = case["params"]
        if p == "mixed":
            settings = dict(temperature=_pick(g, rows, [0.0, 0.6, 0.8, 1.0, 1.3]),
                            top_k=_pick(g, rows, [0, 20, 50, 0], torch.int32),
                            top_p=_pick(g, rows, [1.0, 0.9, 0.95]),
                            min_p=_pick(g, rows, [0.0, 0.0, 0.05]))
        elif p == "top_p":
            settings = dict(temperature=0.8, top_p=0.95)
        elif p == "top_k_top_p":
            settings = dict(temperature=1.0, top_k=64, top_p=0.95)
        elif p == "min_p":
            settings = dict(temperature=1.2, min_p=0.02)
        else:
            settings = dict(temperature=1.0)
        return dict(case=case, logits=logits, uniforms=uniforms, settings=settings)

    vocab, k = case["vocab"], case["k"]
    x = torch.randn(rows, vocab, generator=g, device=DEVICE) * 2.5
    ids = _distinct_ids(g, rows, vocab, k)
    # the teacher's log-probabilities, in candidate order; the student is near them on its good
    # tokens and lower on the others
    steps = torch.arange(k, device=DEVICE) * 0.35
    teacher = -0.5 - steps - 0.2 * _rand(g, rows, k)
    order = torch.argsort(_rand(g, rows, k), dim=1)
    ids = torch.gather(ids, 1, order)
    lift = 14.0 + teacher + 1.5 * torch.randn(rows, k, generator=g, device=DEVICE)
    x.scatter_(1, ids, lift)
    # rows with fewer kept tokens, and rows of padding with none
    kept = torch.where(_rand(g, rows, 1) < 0.1, (_rand(g, rows, 1) * k).long() + 1, k)
    kept = torch.where(_rand(g, rows, 1) < 0.03, 0, kept)
    ids = torch.where(torch.arange(k, device=DEVICE) < kept, ids, -1).to(torch.int32)
    student = x.to(_torch_dtype(case))
    grad_loss = torch.where(kept[:, 0] > 0, 1.0, 0.0) / rows
    state = dict(case=case, student=student, ids=ids.contiguous(), teacher=teacher.contiguous(),
                 grad_loss=grad_loss.float().contiguous())
    if case["direction"] == "backward":
        # what the forward pass keeps: the row's maximum and its sum of exp((z - max) / T)
        f = student.float()
        top = f.amax(dim=1)
        total = torch.zeros(rows, device=DEVICE)
        for r in range(0, rows, 256):
            e = torch.exp((f[r:r + 256].double() - top[r:r + 256, None].double())
                          / case["temperature"])
            total[r:r + 256] = e.sum(dim=1).float()
        state["row_stats"] = torch.stack([top, total], dim=1).contiguous()
    return state


# ---- one pass ----------------------------------------------------------------------------------

def run(state):
    if state["case"]["op"] == "sample":
        return _sample_own(state) if own else _sample_plain(state)
    return _distill_own(state) if own else _distill_plain(state)


def _sample_own(state):
    import dflash2_draft_candidate_amd as d2
    token_ids, logprob = d2.sample(state["logits"], state["uniforms"], **state["settings"])
    return dict(token_ids=token_ids, logprob=logprob)


def _distill_own(state):
    import dflash2_draft_candidate_amd as d2
    case = state["case"]
    t = case["temperature"]
    if case["direction"] == "forward":
        loss, row_stats = d2.distill(state["student"], state["ids"], state["teacher"], t)
        return dict(loss=loss)
    if case["direction"] == "backward":
        return dict(grad=d2.distill_backward(state["student"], state["ids"], state["teacher"],
                                             state["row_stats"], state["grad_loss"], t))
    loss, grad = d2.distill_step(state["student"], state["ids"], state["teacher"],
                                 state["grad_loss"], t)
    return dict(loss=loss, grad=grad)


def _column(value, rows, dtype):
    if isinstance(value, torch.Tensor):
        return value.to(dtype)[:, None]
    return torch.full((rows, 1), value, device=DEVICE, dtype=dtype)


def _sample_plain(state):
    """Sort, weigh, cut, draw. The weights and their running sums are in 64 bits: a token's share
    of a flat row is near the rounding of a 32-bit sum."""
    x = state["logits"].float()
    rows, vocab = x.shape
    s = state["settings"]
    temperature = _column(s.get("temperature", 1.0), rows, torch.float64)
    top_k = _column(s.get("top_k", 0), rows, torch.int64)
    top_p = _column(s.get("top_p", 1.0), rows, torch.float32).double()
    min_p = _column(s.get("min_p", 0.0), rows, torch.float32).double()
    if not isinstance(s.get("temperature", 1.0), torch.Tensor):
        temperature = _column(s.get("temperature", 1.0), rows, torch.float32).double()
    x = torch.where(torch.isnan(x), -math.inf, x)
    value, order = torch.sort(x, dim=1, descending=True, stable=True)
    greedy = temperature <= 0
    gap = value.double() - value[:, :1].double()
    weight = torch.exp(gap / torch.where(greedy, 1.0, temperature))
    rank = torch.arange(vocab, device=x.device)
    weight = torch.where((top_k >= 1) & (rank >= top_k), 0.0, weight)
    running = torch.cumsum(weight, dim=1)
    # the first place where the running sum reaches top_p of the whole ends the nucleus
    inside = (running - weight < top_p * running[:, -1:]) | (top_p >= 1)
    keep = (inside & (weight >= min_p)) | (rank == 0)
    keep = keep & ~(greedy & (rank > 0))
    weight = torch.where(keep, weight, 0.0)
    running = torch.cumsum(weight, dim=1)
    whole = running[:, -1:]
    target = state["uniforms"].double()[:, None] * whole
    place = (running <= target).sum(dim=1, keepdim=True)
    place = torch.minimum(place, keep.sum(dim=1, keepdim=True) - 1)
    token_ids = torch.gather(order, 1, place)[:, 0].int()
    logprob = torch.log(torch.gather(weight, 1, place) / whole)[:, 0].float()
    return dict(token_ids=token_ids, logprob=logprob)


def _distill_plain(state):
    case = state["case"]
    t = case["temperature"]
    z = state["student"].float()
    ids = state["ids"].long()
    valid = ids >= 0
    some = valid.any(dim=1, keepdim=True)
    safe = torch.where(valid, ids, 0)
    teacher = torch.where(valid, state["teacher"] / t, -math.inf)
    top = torch.where(some, teacher.amax(dim=1, keepdim=True), 0.0)
    share = torch.exp(teacher - top)
    share = share / torch.where(some, share.sum(dim=1, keepdim=True), 1.0)
    if case["direction"] == "backward":
        high = state["row_stats"][:, :1]
        e = torch.exp((z - high) / t)
        total = state["row_stats"][:, 1:]
    else:
        high = z.amax(dim=1, keepdim=True)
        e = torch.exp((z - high) / t)
        total = e.sum(dim=1, keepdim=True)
    out = {}
    if case["direction"] != "backward":
        log_q = (torch.gather(z, 1, safe) - high) / t - torch.log(total)
        log_p = torch.log(torch.where(share > 0, share, 1.0))
        term = torch.where(share > 0, share * (log_p - log_q), 0.0)
        out["loss"] = t * t * term.sum(dim=1)
    if case["direction"] != "forward":
        grad = e / total
        grad.scatter_add_(1, safe, -share)
        scale = torch.where(some, state["grad_loss"][:, None] * t, 0.0)
        out["grad"] = (grad * scale).to(state["student"].dtype)
    return out


# ---- what a pass cannot do without ---------------------------------------------------------------

def work(case):
    rows, vocab = case["rows"], case["vocab"]
    size = 2 if case["dtype"] == "bf16" else 4
    whole = rows * vocab * size
    if case["op"] == "sample":
        # logits and uniforms in, ids and log-probabilities out; a weight and a sum per element
        settings = {"mixed": 16 * rows}.get(case["params"], 0)
        return dict(bytes=whole + 12 * rows + settings, flops=4 * rows * vocab)
    small = rows * case["k"] * 8 + 4 * rows
    if case["direction"] == "forward":
        return dict(bytes=whole + small, flops=4 * rows * vocab)
    if case["direction"] == "backward":
        return dict(bytes=2 * whole + small + 8 * rows, flops=4 * rows * vocab)
    return dict(bytes=2 * whole + small + 4 * rows, flops=8 * rows * vocab)


# ---- the definition in 64 bits -------------------------------------------------------------------

def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "sample":
        return _sample_exact(state)
    if case["rows"] * case["vocab"] > 300_000_000:
        return None
    return _distill_exact(state)


def _sample_exact(state):
    """Row by row over the distinct values of the row and how often each occurs."""
    s = state["settings"]
    rows = state["case"]["rows"]

    def setting(name, default):
        v = s.get(name, default)
        if isinstance(v, torch.Tensor):
            return v.tolist()
        if isinstance(v, float):
            v = torch.tensor(v, dtype=torch.float32).item()
        return [v] * rows

    temperature, top_k = setting("temperature", 1.0), setting("top_k", 0)
    top_p, min_p = setting("top_p", 1.0), setting("min_p", 0.0)
    uniforms = state["uniforms"].tolist()
    ids, logs = [], []
    for r in range(rows):
        row = state["logits"][r].double()
        value, count = torch.unique(row, return_counts=True)
        value, count = value.flip(0), count.flip(0)
        if temperature[r] <= 0:
            ids.append(int((row == value[0]).nonzero()[0]))
            logs.append(0.0)
            continue
        w = ((value - value[0]) / temperature[r]).exp()
        n = int(count.sum())
        if 1 <= top_k[r] < n:
            before = count.cumsum(0) - count
            count = (top_k[r] - before).clamp(min=0).minimum(count)
        mass = (w * count).cumsum(0)
        if top_p[r] < 1:
            goal = top_p[r] * mass[-1]
            i = int((mass < goal).sum())
            start = mass[i] - w[i] * count[i]
            need = int(((goal - start) / w[i]).ceil().clamp(min=1))
            count = count[:i + 1].clone()
            count[i] = min(need, int(count[i]))
            w = w[:i + 1]
        kept = (w >= min_p[r])
        kept[0] = True
        w, count = w[kept], count[kept]
        mass = (w * count).cumsum(0)
        goal = uniforms[r] * mass[-1]
        i = min(int((mass <= goal).sum()), len(w) - 1)
        start = mass[i] - w[i] * count[i]
        nth = int(((goal - start) / w[i]).floor().clamp(min=0))
        nth = min(nth, int(count[i]) - 1)
        ids.append(int((row == value[i]).nonzero()[nth]))
        logs.append(float((w[i] / mass[-1]).log()))
    return dict(token_ids=torch.tensor(ids, dtype=torch.int32),
                logprob=torch.tensor(logs, dtype=torch.float64))


def _distill_exact(state):
    case = state["case"]
    t = case["temperature"]
    losses, grads = [], []
    for r in range(case["rows"]):
        z = state["student"][r].double() / t
        pick = state["ids"][r] >= 0
        ids = state["ids"][r][pick].long()
        log_q = z - torch.logsumexp(z, dim=0)
        if len(ids) == 0:
            losses.append(torch.zeros((), device=z.device, dtype=torch.float64))
            grads.append(torch.zeros_like(z))
            continue
        log_p = torch.log_softmax(state["teacher"][r][pick].double() / t, dim=0)
        losses.append(t * t * (log_p.exp() * (log_p - log_q[ids])).sum())
        if case["direction"] != "forward":
            q = log_q.exp()
            q.index_add_(0, ids, -log_p.exp())
            grads.append(q * (t * state["grad_loss"][r].double()))
    out = {}
    if case["direction"] != "backward":
        out["loss"] = torch.stack(losses)
    if case["direction"] != "forward":
        out["grad"] = torch.stack(grads)
    return out
