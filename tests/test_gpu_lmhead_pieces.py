"""The LM head's losses where rows of W are read whole, over more than one piece of the vocabulary; and what
a bad teacher logit reaches (needs an MI355X).

Inputs as multiples of 1/4 and 1/8: logits are exact in fp32 in any order. Tolerances, u = 2^-24:
  * Sigma = sum exp((x - max) / tau). A term's exponent t = (x - max) log2(e) / tau errs by 2 |t| u (the
    rounded coefficient, the rounded product), 128 ln 2 u of the term (|t| <= 64: what lies below counts
    for less than V 2^-64), the hardware exponential by 2 u. Sums are rescaled where a maximum rises: the
    exponents of a chain of rescales add up to at most 64 as well (128 ln 2 u again, and what lies
    below counts for nothing), and each link is an exponential, a product and a sum: 4 u. Links: the tiles of
    8 rows that a workgroup goes through, 3 exchanges of lanes, 256 / 64 partial sums, 6 exchanges.
      eps_sigma = (2 * 128 ln 2 + 2 + 4 (ceil(ceil(V / 8) / 256) + 13)) u
  * loss: tau^2 eps_sigma + u |loss|.
  * G: q by eps_sigma and (128 ln 2 + 6) u (its exponential, g tau / sum, a product); the masses by
    (128 ln 2 + 2 + 6 + 2) u (6 exchanges of the sum, the quotient, the product); the two bf16 parts leave
    2^-16 of it; exp below 2^-100 may be flushed: 1e-30 |g| tau.
  * the products: fp32 sums of n terms, off by at most n 2^-23 sum |G| |W| (the matrix units may truncate
    where they add), n = V + 256 for grad_hidden, 2 R for grad_W; then the rounding to bf16, 2^-8 of the result.
"""
import math
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


def ints(gen, lo, hi, *shape):
    return torch.randint(lo, hi + 1, shape, generator=gen, device=DEV)


@pytest.mark.parametrize("V", [(1 << 20) + 1, (1 << 20) + 70001, (2 << 20) + 9])
@pytest.mark.parametrize("R,H", [(3, 1032), (16, 1032), (20, 1032), (32, 1032)])
def test_whole_rows_in_pieces(d2, R, H, V):
    log(f"lmhead loss whole rows in pieces R={R} H={H} V={V}")
    K, tau = 4, 1.5
    gen = torch.Generator(device=DEV).manual_seed(R + V)
    h = (ints(gen, -5, 5, R, H) / 4).bfloat16()
    W = ((ints(gen, 0, 3, V, H) == 0) * ints(gen, -1, 1, V, H) / 8).bfloat16()
    ids = ints(gen, 0, V - 1, R, K).int()
    edge = 1 << 20
    ids[0] = torch.tensor([0, edge - 1, edge, V - 1])
    ids[1] = torch.tensor([edge, edge, -1, V - 1])
    ids[2, 0] = V
    ids[R - 1] = torch.tensor([edge - 1, 5, edge, 5])
    t = torch.randn(R, K, generator=gen, device=DEV)
    g = torch.randn(R, generator=gen, device=DEV)
    out = None
    if R > 8:
        out = 4
        ids[out] = -1
        h[out] = math.nan
    loss, stats = d2.lmhead_distill(h, W, ids, t, tau)
    gh, gw = d2.lmhead_distill_backward(h, W, ids, t, stats, g, tau)
    only_h, _ = d2.lmhead_distill_backward(h, W, ids, t, stats, g, tau, need_weight=False)
    _, only_w = d2.lmhead_distill_backward(h, W, ids, t, stats, g, tau, need_hidden=False)
    assert torch.equal(only_h, gh) and torch.equal(only_w, gw)
    if out is not None:
        assert float(loss[out]) == 0.0 and bool((gh[out] == 0).all())
        h[out] = 0.0
        g[out] = 0.0
    # 64 bits
    hd, gd = h.double(), g.double()
    x = torch.cat([torch.mm(hd, W[a:a + 400_000].double().t()) for a in range(0, V, 400_000)], dim=1)
    log_q = torch.log_softmax(x / tau, dim=1)
    ok = (ids >= 0) & (ids < V)
    safe = torch.where(ok, ids, 0).long()
    a = torch.where(ok, t.double() / tau, -math.inf)
    if out is not None:
        a[out] = 0.0
    log_p = torch.log_softmax(a, dim=1)
    pj = torch.where(ok, log_p.exp(), 0.0)
    want = tau ** 2 * torch.where(ok, pj * (log_p - log_q.gather(1, safe)), 0.0).sum(dim=1)
    E = 128 * math.log(2)
    sigma = (2 * E + 2 + 4 * (-(-(-(-V // 8)) // 256) + 13)) * U
    assert bool(((loss.double() - want).abs() <= tau ** 2 * sigma + U * want.abs()).all())
    p = torch.zeros_like(x).scatter_add_(1, safe, pj)
    q = log_q.exp()
    s = (gd * tau)[:, None]
    G = s * (q - p)
    dG = s.abs() * (q * (sigma + (E + 6) * U) + p * (E + 10) * U + 1e-30) + 2.0 ** -16 * G.abs()
    aG, hf = G.abs() + dG, 2.0 ** -8
    # all of grad_hidden; grad_W in parts
    wh, th = torch.zeros(R, H, dtype=torch.float64, device=DEV), torch.zeros(R, H, dtype=torch.float64, device=DEV)
    ah = hd.abs()
    for first in range(0, V, 400_000):
        v = slice(first, first + 400_000)
        Wd = W[v].double()
        wh += torch.mm(G[:, v], Wd)
        th += torch.mm((dG + (V + 256) * 2.0 ** -23 * aG)[:, v], Wd.abs())
        ww = torch.mm(G[:, v].t(), hd)
        tol = torch.mm((dG + 2 * R * 2.0 ** -23 * aG)[:, v].t(), ah) * (1 + hf) + hf * ww.abs() + 1e-37
        bad = ~((gw[v].double() - ww).abs() <= tol)
        assert not bool(bad.any()), (first + bad.nonzero()[:4, 0]).tolist()
    tol = th * (1 + hf) + hf * wh.abs() + 1e-37
    bad = ~((gh.double() - wh).abs() <= tol)
    assert not bool(bad.any()), bad.nonzero()[:4].tolist()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("R,H,V", [(14, 1000, 700), (20, 64, 700), (40, 264, 700), (90, 72, 1030), (140, 72, 515),
                                   (400, 136, 515), (14, 1200, 700), (25, 1200, 700), (400, 136, 20001)])
def test_bad_teacher_logits(d2, R, H, V, dt):
    """NaN or +inf among a row's teacher logits: its loss, grad_hidden's row and grad_W at all of the row's
    entries; nothing else."""
    log(f"lmhead loss bad teacher R={R} H={H} V={V} {dt}")
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    gen = torch.Generator(device=DEV).manual_seed(R + V)
    h = (ints(gen, -5, 5, R, H) / 4).to(dtype)
    W = (ints(gen, -1, 1, V, H) / 8).to(dtype)
    for K in (4, 40):
        ids = ints(gen, 0, V - 1, R, K).int()
        t = torch.randn(R, K, generator=gen, device=DEV)
        g = torch.randn(R, generator=gen, device=DEV)
        t[6, 1], t[8, 0] = math.nan, math.inf
        ids[6, 3], ids[8, 2] = -1, V      # no entries; a bad logit there is none either
        ids[9, 0], t[9, 0] = -1, math.nan
        ids[10, 1], t[10, 1] = V, math.inf
        loss, stats = d2.lmhead_distill(h, W, ids, t)
        gh, gw = d2.lmhead_distill_backward(h, W, ids, t, stats, g)
        bad = torch.zeros(R, dtype=torch.bool, device=DEV)
        bad[[6, 8]] = True
        assert torch.equal(torch.isnan(loss), bad) and bool(torch.isfinite(loss[~bad]).all())
        assert bool(torch.isfinite(gh[~bad]).all()) and bool(torch.isnan(gh[bad]).any(dim=1).all())
        named = torch.zeros(V, dtype=torch.bool, device=DEV)
        for r in (6, 8):
            named[ids[r][(ids[r] >= 0) & (ids[r] < V)].long()] = True
        assert bool(torch.isnan(gw[named]).all()) and bool(torch.isfinite(gw[~named]).all())
