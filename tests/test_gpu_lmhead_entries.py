"""The entries' logits of the LM head's losses are the ones in their rows' sums (needs an MI355X).

The loss and the gradient of a row that is sure of its target are small differences: x_target - max,
q_target - 1. They keep their digits where both logits are the same fp32 numbers, however far these are
from the exact ones. Logits here are about 1000, sums of 2048 products and less, which two orders of
summation give up to 1e-4 apart. u = 2^-24.
  * Where a row's target is its maximum, the kept logit is the kept maximum, bit for bit; then loss =
    log(sum) in 64 bits, rounded once.
  * The sum: an exponential's relative error is 128 ln 2 u + 2 u at most (what lies below 2^-64 counts for
    less than V 2^-64), so the terms beside the maximum's, which is 1 exactly, are off by 91 u of their
    total, and their logits by d each, d = H 2^-23 sum |h| |W|: by (e^(2 d) - 1) of it. Every addition to
    the partial sum that holds the 1 rounds by u of it: at most 32 a tile of a lane's columns (3 tiles), 2
    exchanges, 7 waves, ceil(parts / 64) + 6 partial sums: fewer than 128.
  * sum_v G is 0: W's first column is 1 and hidden's 0, so it is grad_hidden's first column. G's values
    err by 192 u in all (four times an exponential's hardware error, the sum's 128 u, what forms g / sum
    and q - p, the products' additions), and bf16 rounds each by 2^-8 of it: 2^-8 sum |G| = 2^-8 2 (1 - 1 / sum)
    for g = 1, and the result once more.
"""
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24


def log(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module")
def d2():
    import dflash2_draft_candidate_amd
    return dflash2_draft_candidate_amd


def inputs(R, H, V, dtype, seed):
    """Rows that are more or less sure (by about 8 to 30) of a token each, among logits of about 1000."""
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    wide = (2048 / H) ** 0.5
    base = randn(H) * wide
    part = randn(V, H) * (0.07 * wide)  # what tokens differ by, at a right angle to base
    W = base + part - (part @ base / (base @ base))[:, None] * base
    top = torch.randint(0, V, (R,), generator=gen, device=DEV)
    top[0], top[-1] = 0, V - 1
    lift = 1.3 + 1.5 * torch.rand(R, 1, generator=gen, device=DEV)
    h = base * 0.5 + randn(R, H) * (0.1 * wide) + (W[top] - base) * lift
    h[:, 0], W[:, 0] = 0.0, 1.0
    return h.to(dtype), W.to(dtype), top.int()


# every way through the kernels: rows of W read whole, rings that find the entries, rings behind a gather,
# streams
WAYS = [(5, 264), (5, 2048), (25, 2048), (32, 520), (64, 264), (64, 2048), (65, 264), (65, 2056), (100, 1016),
        (128, 2048), (129, 264), (331, 2048), (600, 1032)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("R,H", WAYS)
def test_one_token(d2, R, H, dt):
    """A vocabulary of one: the entry's logit is the maximum, the sum is 1, the loss 0."""
    log(f"lmhead entries, one token R={R} H={H} {dt}")
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    h, W, top = inputs(R, H, 1, dtype, R + H)
    loss, stats = d2.lmhead_ce(h, W, top)
    assert float(stats[:, 0].abs().max()) > 500.0
    assert torch.equal(stats[:, 0], stats[:, 2])
    assert bool((stats[:, 1] == 1).all()) and bool((loss == 0).all())
    for K in (3, 33):
        ids = torch.zeros(R, K, dtype=torch.int32, device=DEV)
        ids[:, 1] = -1
        loss, stats = d2.lmhead_distill(h, W, ids, torch.zeros(R, K, device=DEV))
        assert torch.equal(stats[:, 0], stats[:, 2]) and torch.equal(stats[:, 0], stats[:, 1 + K])
        assert bool((stats[:, 3] == 0).all())


@pytest.mark.parametrize("V", [16, 257, 700])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("R,H", WAYS)
def test_sure_rows(d2, R, H, V, dt):
    log(f"lmhead entries, sure rows R={R} H={H} V={V} {dt}")
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    h, W, top = inputs(R, H, V, dtype, R + H + V)
    x = torch.mm(h.double(), W.double().t())
    first, second = x.topk(2, dim=1).values.t()
    assert bool((x.argmax(dim=1) == top).all()) and float((first - second).min()) > 1.0
    exact = torch.logsumexp(x, dim=1) - first
    assert float(exact.min()) < 1e-3
    loss, stats = d2.lmhead_ce(h, W, top)
    assert torch.equal(stats[:, 0], stats[:, 2])
    s = stats[:, 1].double()
    assert bool(((loss.double() - s.log()).abs() <= U * s.log()).all())
    d = H * 2.0 ** -23 * torch.mm(h.double().abs(), W.double().abs().t()).amax(dim=1)
    lim = (torch.expm1(2 * d) + 92 * U) * torch.expm1(exact) + 129 * U
    assert bool(((loss.double() - exact).abs() <= lim).all())
    # the same loss as a teacher's with one entry of all the mass, among others without
    K = 5
    ids = torch.randint(0, V, (R, K), device=DEV).int()
    t = torch.full((R, K), -float("inf"), device=DEV)
    ids[:, 3], t[:, 3] = top, 0.5
    again, more = d2.lmhead_distill(h, W, ids, t)
    assert torch.equal(again, loss) and torch.equal(more[:, 5], stats[:, 0])
    # many entries, the sure one behind them
    K = 40
    ids = torch.randint(0, V, (R, K), device=DEV).int()
    ids[:, K - 1] = top
    _, more = d2.lmhead_distill(h, W, ids, torch.zeros(R, K, device=DEV))
    assert torch.equal(more[:, 2:].amax(dim=1), more[:, 0])
    # sum_v G
    gh, _ = d2.lmhead_ce_backward(h, W, top, stats, torch.ones(R, device=DEV), need_weight=False)
    off = 2 * (1 - 1 / s) * (2.0 ** -8 if dtype == torch.bfloat16 else 0.0)
    half = 2.0 ** -8 if dtype == torch.bfloat16 else U
    assert bool((gh[:, 0].double().abs() <= (off + 192 * U) * (1 + half)).all())
