"""The gradients of more than 64 bf16 rows keep what rounding G to bf16 leaves of its values at the entries,
those of a 32nd of the row's largest mass and more (needs an MI355X).

Inputs are multiples of 1/4 and 1/8 (logits are exact in fp32 in any order), and all columns but a few lie 300
below these: their q is 0, and G with it. So G is not 0 at the few columns alone, which all rows name
(distillation), or at two, of which all rows name the same one (cross entropy: grad_W's row of that one is what
is compared). Some 40 rows have a grad_loss that is not 0. With u = 2^-24, E = 128 ln 2:
  * q: the sum's terms err by (E + 2) u, its rescales' exponents add up to E u, and each of at most 64 links of
    the chain of partial sums is an exponential, a product and a sum, 4 u, with 32 additions before them:
    eps_sigma = (2 E + 2 + 256 + 32) u; its own exponential, the quotient and the product (E + 6) u more; the masses
    (E + 2 + 6 + 2) u.
  * G in two bf16 parts: 2^-16 of it; terms below 2^-100 may be flushed: 1e-30 |g| tau.
  * the products: fp32 sums of n terms that are not 0, off by n 2^-23 of their magnitudes (the matrix units may
    truncate where they add): two parts of the columns for grad_hidden, of the 40 rows for grad_W; then the rounding
    to bf16, 2^-8 of the result.
One part alone is off by up to 2^-8 of each G, far more where the sums are small.
"""
import math
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
E = 128 * math.log(2)
SIGMA = (2 * E + 2 + 256 + 32) * U


def log(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module")
def d2():
    import dflash2_draft_candidate_amd
    return dflash2_draft_candidate_amd


def ints(gen, lo, hi, *shape):
    return torch.randint(lo, hi + 1, shape, generator=gen, device=DEV)


def inputs(R, H, V, at, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    h = (ints(gen, -5, 5, R, H) / 4).bfloat16()
    W = (ints(gen, -1, 1, V, H) / 8).bfloat16()
    W[:, 0] = -300.0
    W[at, 0] = 0.0
    h[:, 0] = 1.0
    g = torch.zeros(R, device=DEV)
    some = torch.randperm(R, generator=gen, device=DEV)[:38]
    g[some] = torch.randn(some.numel(), generator=gen, device=DEV)
    g[0], g[-1] = 0.7, -1.3
    out = torch.zeros(R, dtype=torch.bool, device=DEV)
    out[5::7] = True
    out[0] = out[-1] = False
    h[out] = math.nan
    g[out] = math.nan
    return gen, h, W, g, out


def compare(h, W, g, out, at, p, got_h, got_w, tau, columns):
    """p: the masses at the columns `at`; columns: of `at`, those of grad_W to compare (all others of grad_W
    are 0)."""
    hd, Ws = torch.where(out[:, None], 0.0, h).double(), W[at].double()
    s = torch.where(out, 0.0, g).double()[:, None] * tau
    q = torch.softmax(torch.mm(hd, Ws.t()) / tau, dim=1)
    G = s * (q - p)
    dG = s.abs() * (q * (SIGMA + (E + 6) * U) + p * (E + 10) * U + 1e-30) + 2.0 ** -16 * G.abs()
    aG, hf = G.abs() + dG, 2.0 ** -8
    n = at.numel()
    if columns is None:  # (grad_hidden too)
        want = torch.mm(G, Ws)
        tol = torch.mm(dG + 2 * n * 2.0 ** -23 * aG, Ws.abs()) * (1 + hf) + hf * want.abs() + 1e-37
        bad = ~((got_h.double() - want).abs() <= tol)
        assert not bool(bad.any()), ("grad_hidden", int(bad.sum()), bad.nonzero()[:4].tolist())
        columns = torch.arange(n, device=DEV)
    want = torch.mm(G.t(), hd)
    tol = torch.mm((dG + 2 * 40 * 2.0 ** -23 * aG).t(), hd.abs()) * (1 + hf) + hf * want.abs() + 1e-37
    bad = ~((got_w[at].double() - want).abs() <= tol)[columns]
    assert not bool(bad.any()), ("grad_W", int(bad.sum()), bad.nonzero()[:4].tolist())
    rest = torch.ones(W.shape[0], dtype=torch.bool, device=DEV)
    rest[at] = False
    assert bool((got_w[rest] == 0).all())


SIZES = [(65, 64, 64), (65, 1000, 700), (100, 2056, 3001), (128, 264, 64), (128, 4104, 1000), (129, 200, 700),
         (200, 1000, 2049), (256, 264, 513), (257, 264, 513), (331, 136, 20001), (600, 2056, 1500),
         (700, 64, 300), (1024, 72, 140001), (3000, 64, 30001), (5000, 72, 1100), (65536, 8, 20001), (65536, 8, 900)]


@pytest.mark.parametrize("R,H,V", SIZES)
@pytest.mark.parametrize("n,near", [(1, False), (3, False), (14, False), (14, True), (61, True), (61, False)])
def test_entries_in_two_parts(d2, R, H, V, n, near):
    """n columns that all rows name, side by side or anywhere, and one of them twice, and no column."""
    if n > V - 2:
        n = V // 2
    log(f"lmhead precision R={R} H={H} V={V} n={n} near={near}")
    tau = 1.25
    first = torch.randperm(V, generator=torch.Generator().manual_seed(n + R))[:n].sort().values.to(DEV)
    at = V - n + torch.arange(n, device=DEV) if near else first
    if not near and n > 2:
        at[0], at[-1] = 0, V - 1
    gen, h, W, g, out = inputs(R, H, V, at, R + V + n)
    ids = at[torch.rand(R, n, generator=gen, device=DEV).argsort(dim=1)].int()
    ids = torch.cat([ids, ids[:, :1], torch.full((R, 1), V, device=DEV, dtype=torch.int32)], dim=1).contiguous()
    t = 4.0 * torch.rand(R, n + 2, generator=gen, device=DEV)  # (masses within a 32nd: e^(4 / 1.25) < 32)
    ids[out] = -1
    loss, stats = d2.lmhead_distill(h, W, ids, t, tau)
    gh, gw = d2.lmhead_distill_backward(h, W, ids, t, stats, g, tau)
    only_h, _ = d2.lmhead_distill_backward(h, W, ids, t, stats, g, tau, need_weight=False)
    _, only_w = d2.lmhead_distill_backward(h, W, ids, t, stats, g, tau, need_hidden=False)
    assert torch.equal(gh, only_h) and torch.equal(gw, only_w)
    mass = torch.softmax(t[:, :n + 1].double() / tau, dim=1)
    place = torch.searchsorted(at, torch.where(out[:, None], at[:1], ids[:, :n + 1].long()))
    p = torch.zeros(R, n, dtype=torch.float64, device=DEV).scatter_add_(1, place, mass)
    compare(h, W, g, out, at, p, gh, gw, tau, None)


@pytest.mark.parametrize("R,H,V", SIZES)
def test_target_in_two_parts(d2, R, H, V):
    log(f"lmhead precision, targets R={R} H={H} V={V}")
    at = torch.tensor([V // 3, V - 1], device=DEV)
    gen, h, W, g, out = inputs(R, H, V, at, R + V)
    targets = torch.where(out, -1, V - 1).int()
    loss, stats = d2.lmhead_ce(h, W, targets)
    gh, gw = d2.lmhead_ce_backward(h, W, targets, stats, g)
    p = torch.zeros(R, 2, dtype=torch.float64, device=DEV)
    p[:, 1] = 1.0
    compare(h, W, g, out, at, p, gh, gw, 1.0, torch.tensor([1], device=DEV))


@pytest.mark.parametrize("R,H,V", [(100, 264, 3001), (300, 264, 3001), (1024, 72, 140001)])
def test_graph_replay(d2, R, H, V):
    """Lists of other lengths on every replay, none among them."""
    log(f"lmhead precision graph R={R}")
    sets = []
    for i in range(3):
        at = torch.arange(i, V, 1 + V // 9, device=DEV)
        gen, h, W, g, out = inputs(R, H, V, at, i)
        ids = at[ints(gen, 0, at.numel() - 1, R, 4)].int()
        ids[out] = -1
        if i == 2:
            ids[:] = -1
        sets.append((h, W, ids, torch.randn(R, 4, generator=gen, device=DEV), torch.where(out, 0.0, g)))
    buf = [x.clone() for x in sets[0]]

    def step(h, W, ids, t, g):
        loss, stats = d2.lmhead_distill(h, W, ids, t)
        return (loss, *d2.lmhead_distill_backward(h, W, ids, t, stats, g))

    step(*buf)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*buf)
    for i in (0, 1, 2, 0, 1):
        for x, y in zip(buf, sets[i]):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        want = step(*sets[i])
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
