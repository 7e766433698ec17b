"""Measured cases of the operators of a drafter's training step, from hidden states on.

ce        softmax cross entropy of the LM head's product with given target tokens, and the
          gradients of the hidden states and of the head's weight, without the logits.
distill   the same from a teacher's top logits (a loss the package has for given logits).
clip      the global norm over a step's gradients, and the gradients clipped by it.

A case is a plain dict; `run` computes it in elementary torch operations, or, where `own` is
true, through the package's entry points.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"

# Vocabularies, hidden sizes and row counts are those of the selector's workloads (a draft block
# of 16 positions; 64 sequences, 32 sequences of the larger vocabulary) and generic odd ones.
# `grads`: none (an evaluation), hidden (the head is frozen: a drafter shares its target's) or
# both. `ignored`: share of the rows that have no target (prompts, padding).


def listed():
    return [
        # the loss of one draft block, as an evaluation asks for it
        dict(name="ce-loss-block", op="ce", rows=16, hidden=4096, vocab=151936, dtype="bf16",
             grads="none", ignored=0.0),
        # one draft block trained on, head and all
        dict(name="ce-train-block", op="ce", rows=16, hidden=4096, vocab=151936, dtype="bf16",
             grads="both", ignored=0.1),
        # small model, float32, sizes that fit no tile
        dict(name="ce-train-f32-odd", op="ce", rows=331, hidden=1016, vocab=32003, dtype="f32",
             grads="both", ignored=0.1),
        # a small vocabulary, few rows: launches count
        dict(name="ce-train-small", op="ce", rows=40, hidden=256, vocab=1024, dtype="bf16",
             grads="both", ignored=0.1),
        # 64 draft blocks trained on
        dict(name="ce-train-1024", op="ce", rows=1024, hidden=4096, vocab=151936, dtype="bf16",
             grads="both", ignored=0.0),
        # a large step: 256 draft blocks, a quarter of the rows without a target
        dict(name="ce-train-4096", op="ce", rows=4096, hidden=4096, vocab=151936, dtype="bf16",
             grads="both", ignored=0.25),
        # the loss alone, odd sizes
        dict(name="distill-loss-odd", op="distill", rows=77, hidden=1032, vocab=50021, k=7,
             dtype="bf16", temperature=1.5, grads="none", ignored=0.05),
        # 32 draft blocks of the larger vocabulary, frozen head
        dict(name="distill-frozen-512", op="distill", rows=512, hidden=5376, vocab=262144, k=16,
             dtype="bf16", temperature=1.0, grads="hidden", ignored=0.03),
        # 64 draft blocks, head trained too
        dict(name="distill-train-1024", op="distill", rows=1024, hidden=4096, vocab=151936, k=64,
             dtype="bf16", temperature=2.0, grads="both", ignored=0.03),
        # the convolution's kernels alone: a few short tensors, launches count
        dict(name="clip-kernels", op="clip", tensors="kernels", count=20, clip=True),
        # many odd tensors of both types, views that start anywhere
        dict(name="clip-ragged", op="clip", tensors="ragged", count=400, largest=2_000_000,
             clip=True),
        # the selector's tensors and a drafter's layers
        dict(name="clip-drafter", op="clip", tensors="drafter", count=5, clip=True),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ce", "ce", "distill", "distill", "clip"])
    if op == "clip":
        kind = rng.choice(["kernels", "ragged", "ragged", "drafter"])
        if kind == "ragged":
            return dict(op=op, tensors=kind, count=_log_uniform(rng, 1, 600),
                        largest=_log_uniform(rng, 10, 2_500_000), clip=rng.random() < 0.7)
        most = 64 if kind == "kernels" else 5
        return dict(op=op, tensors=kind, count=rng.randint(1, most), clip=rng.random() < 0.7)
    vocab = _log_uniform(rng, 1000, 262144)
    if rng.random() < 0.5:
        vocab |= 1
    hidden = 8 * _log_uniform(rng, 8, 672)
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    # no more than the largest listed case in either type's products
    most = min(4096, 2_500_000_000_000 // (vocab * hidden) // (1 if dtype == "bf16" else 4))
    case = dict(op=op, rows=_log_uniform(rng, 1, most), hidden=hidden, vocab=vocab, dtype=dtype,
                grads=rng.choice(["none", "hidden", "both", "both"]),
                ignored=rng.choice([0.0, 0.05, 0.3]))
    if op == "distill":
        case.update(k=_log_uniform(rng, 1, 64), temperature=rng.choice([0.75, 1.0, 1.5, 2.0]))
    return case


# ---- inputs ------------------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device=DEVICE)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEVICE)


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "clip":
        return _prepare_clip(case, g)
    rows, hidden, vocab = case["rows"], case["hidden"], case["vocab"]
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    # logits of spread 3, as the selector's workloads have them
    weight = (_randn(g, vocab, hidden) * (3.0 / math.sqrt(hidden))).to(dtype)
    h = _randn(g, rows, hidden)
    keep = _rand(g, rows) >= case["ignored"]
    # tokens of the text: a few are frequent
    k = case.get("k", 1)
    part = vocab // k
    ids = torch.arange(k, device=DEVICE) * part + (_rand(g, rows, k) ** 3 * part).long()
    # the model has learned something: its hidden states point to the target, more or less
    lift = (4.0 * _rand(g, rows, 1)) / 3.0
    h = (h + lift * weight[ids[:, 0]].float()).to(dtype)
    state = dict(case=case, hidden=h.contiguous(), weight=weight,
                 grad_loss=(torch.where(keep, 0.5 + _rand(g, rows), 0.0) / rows).contiguous())
    if case["op"] == "ce":
        state["targets"] = torch.where(keep, ids[:, 0], -1).int().contiguous()
        return state
    teacher = -0.5 - 0.35 * torch.arange(k, device=DEVICE) - 0.2 * _rand(g, rows, k)
    kept = torch.where(_rand(g, rows, 1) < 0.1, (_rand(g, rows, 1) * k).long() + 1, k)
    kept = torch.where(keep[:, None], kept, 0)
    state["ids"] = torch.where(torch.arange(k, device=DEVICE) < kept, ids, -1).int().contiguous()
    state["teacher"] = teacher.contiguous()
    return state


def _clip_shapes(case):
    """(shape, type, elements before it in its storage) of each gradient; a case's own, the same
    for every seed."""
    bf16, f32 = torch.bfloat16, torch.float32
    n = case["count"]
    if case["tensors"] == "kernels":
        return [((2, 4096), bf16, 0) for _ in range(n)]
    if case["tensors"] == "drafter":
        out = [((4096, 64), bf16, 0), ((151936, 64), bf16, 0), ((151936, 64), bf16, 0)]
        for _ in range(n):
            out += [((4096, 4096), bf16, 0)] * 4 + [((12288, 4096), bf16, 0)] * 3
            out += [((4096,), f32, 0)] * 2 + [((2, 4096), bf16, 0)] * 4
        return out
    rng = random.Random(n * 1_000_003 + case["largest"])
    return [((_log_uniform(rng, 1, case["largest"]),), rng.choice([bf16, bf16, f32]),
             rng.randrange(8)) for _ in range(n)]


def _flat_places(case):
    """Where each gradient's result stands in the flat buffer of its type, and the buffers' sizes."""
    places, ends = [], {torch.bfloat16: 0, torch.float32: 0}
    for shape, dtype, before in _clip_shapes(case):
        first = ends[dtype] + before
        places.append((dtype, first, first + math.prod(shape)))
        ends[dtype] = first + math.prod(shape)
    return places, {d: n for d, n in ends.items() if n > 0}


def _prepare_clip(case, g):
    """The gradients, each in a storage of its own, and the flat buffers (one a type, as an
    optimizer keeps them) that the clipped ones go to."""
    grads, outs = [], []
    places, sizes = _flat_places(case)
    flats = {d: torch.zeros(n, dtype=d, device=DEVICE) for d, n in sizes.items()}
    for i, ((shape, dtype, before), (_, first, last)) in enumerate(zip(_clip_shapes(case),
                                                                       places)):
        n = math.prod(shape)
        whole = (_randn(g, n + before) * (0.002 * (1 + i % 7))).to(dtype)
        grads.append(whole[before:].view(shape))
        outs.append(flats[dtype][first:last].view(shape))
    return dict(case=case, grads=grads, outs=outs, flats=list(flats.values()), max_norm=1.0)


# ---- one pass ----------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if op == "clip":
        return _clip_own(state) if own else _clip_plain(state)
    return _loss_own(state) if own else _loss_plain(state)


def _loss_own(state):
    import dflash2_draft_candidate_amd as d2
    case = state["case"]
    h, w = state["hidden"], state["weight"]
    if case["op"] == "ce":
        side = (state["targets"],)
        loss, row_stats = d2.lmhead_ce(h, w, *side)
        backward, more = d2.lmhead_ce_backward, {}
    else:
        side = (state["ids"], state["teacher"])
        more = dict(temperature=case["temperature"])
        loss, row_stats = d2.lmhead_distill(h, w, *side, **more)
        backward = d2.lmhead_distill_backward
    out = dict(loss=loss)
    if case["grads"] != "none":
        out["grad_hidden"], grad_w = backward(h, w, *side, row_stats, state["grad_loss"],
                                              need_weight=case["grads"] == "both", **more)
        if case["grads"] == "both":
            out["grad_weight"] = grad_w
    return out


def _clip_own(state):
    import dflash2_draft_candidate_amd as d2
    if not state["case"]["clip"]:
        return dict(norm=d2.grad_norm(state["grads"]))
    norm = d2.clip_grads(state["grads"], state["max_norm"], out=state["outs"])
    return dict(norm=norm, grads=state["flats"])


def _loss_plain(state):
    case = state["case"]
    h, w = state["hidden"].float(), state["weight"].float()
    t = case.get("temperature", 1.0)
    if case["op"] == "ce":
        ids = state["targets"].long()[:, None]
        teacher = torch.zeros(ids.shape, device=h.device)
    else:
        ids, teacher = state["ids"].long(), state["teacher"]
    valid = ids >= 0
    some = valid.any(dim=1, keepdim=True)
    safe = torch.where(valid, ids, 0)
    teacher = torch.where(valid, teacher / t, -math.inf)
    share = torch.exp(teacher - torch.where(some, teacher.amax(dim=1, keepdim=True), 0.0))
    share = share / torch.where(some, share.sum(dim=1, keepdim=True), 1.0)
    x = h @ w.t()
    picked = torch.gather(x, 1, safe)
    high = x.amax(dim=1, keepdim=True)
    e = torch.exp((x - high) / t)
    del x
    total = e.sum(dim=1, keepdim=True)
    log_q = (picked - high) / t - torch.log(total)
    log_p = torch.log(torch.where(share > 0, share, 1.0))
    term = torch.where(share > 0, share * (log_p - log_q), 0.0)
    out = dict(loss=t * t * term.sum(dim=1))
    if case["grads"] != "none":
        grad = e.div_(total)
        grad.scatter_add_(1, safe, -share)
        grad.mul_(torch.where(some, state["grad_loss"][:, None] * t, 0.0))
        out["grad_hidden"] = (grad @ w).to(state["hidden"].dtype)
        if case["grads"] == "both":
            out["grad_weight"] = (grad.t() @ h).to(state["weight"].dtype)
    return out


def _clip_plain(state):
    squares = [g.float().square().sum(dtype=torch.float64) for g in state["grads"]]
    norm = torch.stack(squares).sum().sqrt()
    if not state["case"]["clip"]:
        return dict(norm=norm.float())
    factor = (state["max_norm"] / torch.clamp(norm, min=state["max_norm"])).float()
    for g, o in zip(state["grads"], state["outs"]):
        o.copy_(g.float() * factor)
    return dict(norm=norm.float(), grads=state["flats"])


# ---- what a pass cannot do without ---------------------------------------------------------------

def work(case):
    if case["op"] == "clip":
        shapes = _clip_shapes(case)
        total = sum(math.prod(s) * (2 if d == torch.bfloat16 else 4) for s, d, _ in shapes)
        elements = sum(math.prod(s) for s, _, _ in shapes)
        if case["clip"]:
            return dict(bytes=2 * total, flops=3 * elements)
        return dict(bytes=total, flops=2 * elements)
    size = 2 if case["dtype"] == "bf16" else 4
    rows, hidden, vocab = case["rows"], case["hidden"], case["vocab"]
    inputs = (rows + vocab) * hidden * size + rows * 8 * case.get("k", 1) + 4 * rows
    product = 2 * rows * hidden * vocab
    grad_hidden, grad_weight = rows * hidden * size, vocab * hidden * size
    if case["grads"] == "none":
        return dict(bytes=inputs, flops=product)
    if case["grads"] == "hidden":
        return dict(bytes=inputs + grad_hidden, flops=2 * product)
    return dict(bytes=inputs + grad_hidden + grad_weight, flops=3 * product)


# ---- the definition in 64 bits -------------------------------------------------------------------

def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "clip":
        return _clip_exact(state)
    return _loss_exact(state)


def _clip_exact(state):
    norm = math.sqrt(math.fsum(float((g.double() ** 2).sum()) for g in state["grads"]))
    out = dict(norm=torch.tensor(norm, dtype=torch.float64))
    if state["case"]["clip"]:
        factor = min(1.0, state["max_norm"] / norm) if norm > 0 else 1.0
        places, sizes = _flat_places(state["case"])
        flats = {d: torch.zeros(n, dtype=torch.float64, device=DEVICE) for d, n in sizes.items()}
        for g, (dtype, first, last) in zip(state["grads"], places):
            flats[dtype][first:last] = g.double().flatten() * factor
        out["grads"] = list(flats.values())
    return out


def _loss_exact(state):
    """Groups of rows, each with its whole softmax."""
    case = state["case"]
    w = state["weight"].double()
    tau = case.get("temperature", 1.0)
    losses, grads_h = [], []
    grad_w = torch.zeros_like(w) if case["grads"] == "both" else None
    group = max(1, 300_000_000 // case["vocab"])
    for first in range(0, case["rows"], group):
        rows = slice(first, first + group)
        h = state["hidden"][rows].double()
        log_q = torch.log_softmax(torch.mm(h, w.T) / tau, dim=1)
        n = h.shape[0]
        p = torch.zeros_like(log_q)
        entropy = torch.zeros(n, dtype=torch.float64, device=w.device)
        if case["op"] == "ce":
            r = (state["targets"][rows] >= 0).nonzero()[:, 0]
            p[r, state["targets"][rows][r].long()] = 1.0
        else:
            logits = state["teacher"][rows].double() / tau
            logits[state["ids"][rows] < 0] = -math.inf
            for r in range(n):
                named = state["ids"][rows][r] >= 0
                if bool(named.any()):
                    lp = torch.log_softmax(logits[r][named], dim=0)
                    p[r].index_add_(0, state["ids"][rows][r][named].long(), lp.exp())
                    entropy[r] = (lp.exp() * lp).sum()
        losses.append(tau * tau * (entropy - (p * log_q).sum(dim=1)))
        if case["grads"] != "none":
            active = p.sum(dim=1) > 0
            d = (log_q.exp() - p) * (tau * state["grad_loss"][rows].double() * active)[:, None]
            grads_h.append(torch.mm(d, w))
            if grad_w is not None:
                grad_w += torch.mm(d.T, h)
    out = dict(loss=torch.cat(losses))
    if case["grads"] != "none":
        out["grad_hidden"] = torch.cat(grads_h)
    if grad_w is not None:
        out["grad_weight"] = grad_w
    return out
