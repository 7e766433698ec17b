"""Cross entropy and distillation of the LM head's product vs a plain implementation in 64 bits
(needs an MI355X).

Inputs are small multiples of 1/4 (hidden) and 1/8 (W), so every product and every partial sum of a
logit is a multiple of 1/32 below 2^18: fp32 holds it exactly in any order, and so do the maxima and
the differences x - max. Tolerances then come from what follows, with u = 2^-24 (half a step of
fp32, relative) and t = (x - max) log2(e) / tau:
  * Sigma = sum exp((x - max) / tau): a term's exponent errs by the rounding of log2(e) / tau and of
    the product, at most 2 |t| u, which is 2 |t| u ln 2 of the term (|t| <= 64: what lies below
    counts for less than V 2^-64), the hardware exponential by 2 u. A lane adds at most 32 terms of
    a tile, two exchanges join 4 lanes; the tiles' pairs are joined in a chain of at most
    ceil(parts / 32), parts = 8 ceil(V / 256), and 5 more, each a rescale by a rounded exponential (its
    exponent errs as above), a product and a sum.
      eps_sigma = (E + 34 + J (E + 3)) u,  E = 128 ln 2 + 2,  J = ceil(parts / 32) + 5
  * loss: what follows is fp64, then one rounding: tau^2 eps_sigma + u |loss|.
  * G: q = exp / Sigma: eps_q = eps_sigma + (E + 4) u (coefficient and products); the entries' masses
    p: eps_p = (E + 2 + 64 + 4) u; |g| tau (q eps_q + p eps_p), and the rounding to the type: 2^-8 of
    G in bf16, u in f32. exp below 2^-100 may be flushed: 1e-30 |g| tau.
  * the products: fp32 sums of n terms, off by at most n 2^-23 sum |G| |W| (the matrix units may
    truncate where they add), n = V (+ pieces and splits: 64) for grad_hidden and R for grad_W; then
    the rounding to the type, 2^-8 or u of the result.
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


def half(dtype):
    return U if dtype == torch.float32 else 2.0 ** -8


def eps(V):
    E = 128 * math.log(2) + 2
    J = -(-8 * -(-V // 256) // 32) + 5
    sigma = (E + 34 + J * (E + 3)) * U
    return sigma, sigma + (E + 4) * U, (E + 70) * U


def reference(h, W, ids, t, g, tau):
    """loss, G, q and p (per vocabulary entry) in 64 bits. t None: a target token per row."""
    h, W, g = h.double(), W.double(), g.double()
    if t is None:
        ids, t = ids[:, None], torch.zeros(ids.shape[0], 1, device=h.device)
    ids, t = ids.long(), t.double()
    R, V = h.shape[0], W.shape[0]
    ok = (ids >= 0) & (ids < V)
    a = torch.where(ok, t / tau, -math.inf)
    active = ((a > -math.inf) | torch.isnan(a)).any(dim=1)
    hz = torch.where(active[:, None], h, 0.0)
    log_q = torch.log_softmax(torch.mm(hz, W.t()) / tau, dim=1)
    q = log_q.exp()
    a = torch.where(active[:, None], a, 0.0)
    log_p = torch.log_softmax(a, dim=1)
    pj = torch.where(ok & active[:, None], log_p.exp(), 0.0)
    safe = torch.where(ok, ids, 0)
    term = torch.where(pj == 0, 0.0, pj * (log_p - log_q.gather(1, safe)))
    loss = torch.where(active, tau * tau * term.sum(dim=1), 0.0)
    p = torch.zeros(R, V, dtype=torch.float64, device=h.device).scatter_add_(1, safe, pj)
    s = torch.where(active, g * tau, 0.0)[:, None]
    return dict(loss=loss, G=s * (q - p), q=q * active[:, None], p=p, s=s.abs(), active=active,
                h=hz, W=W)


def check(ref, loss, gh, gw, dtype, tau, rows=None):
    """rows: those to compare (grad_W not compared then)."""
    R, V = ref["G"].shape
    rows = torch.arange(R, device=DEV) if rows is None else rows
    sigma, eps_q, eps_p = eps(V)
    want = ref["loss"][rows]
    err = (loss.double()[rows] - want).abs()
    assert bool((err <= tau * tau * sigma + U * want.abs()).all()), float(err.max())
    hf = half(dtype)
    dG = ref["s"] * (ref["q"] * eps_q + ref["p"] * eps_p + 1e-30) * (1 + hf) + hf * ref["G"].abs()
    aG = ref["G"].abs() + dG
    if gh is not None:
        want = torch.mm(ref["G"], ref["W"])
        tol = torch.mm(dG, ref["W"].abs()) + (V + 64) * 2.0 ** -23 * torch.mm(aG, ref["W"].abs())
        tol = tol * (1 + hf) + hf * want.abs() + 1e-37
        err = (gh.double() - want).abs()
        bad = ~(err <= tol)[rows]
        assert not bool(bad.any()), (bad.nonzero()[:4], float((err / tol)[rows].max()))
    if gw is not None:
        want = torch.mm(ref["G"].t(), ref["h"])
        tol = torch.mm(dG.t(), ref["h"].abs()) + R * 2.0 ** -23 * torch.mm(aG.t(), ref["h"].abs())
        tol = tol * (1 + hf) + hf * want.abs() + 1e-37
        err = (gw.double() - want).abs()
        bad = ~(err <= tol)
        assert not bool(bad.any()), (bad.nonzero()[:4], float((err / tol).max()))


def inputs(R, H, V, K, dtype, seed):
    """K 0: target tokens."""
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi + 1, shape, generator=gen, device=DEV)

    h = (ints(-5, 5, R, H) / 4).to(dtype)
    wide = max(1, round(24 / math.sqrt(H)))  # logits of a spread of a few
    W = (ints(-wide, wide, V, H) / 8).to(dtype)
    n = max(K, 1)
    ids = torch.randint(0, V, (R, n), generator=gen, device=DEV).int()
    g = torch.randn(R, generator=gen, device=DEV)
    if K == 0:
        return h, W, ids[:, 0].contiguous(), None, g
    t = torch.randn(R, K, generator=gen, device=DEV) * 2
    return h, W, ids, t, g


def forward(d2, h, W, ids, t, tau):
    return d2.lmhead_ce(h, W, ids) if t is None else d2.lmhead_distill(h, W, ids, t, tau)


def backward(d2, h, W, ids, t, stats, g, tau, **need):
    if t is None:
        return d2.lmhead_ce_backward(h, W, ids, stats, g, **need)
    return d2.lmhead_distill_backward(h, W, ids, t, stats, g, tau, **need)


def run(d2, h, W, ids, t, g, tau):
    loss, stats = forward(d2, h, W, ids, t, tau)
    return (loss, *backward(d2, h, W, ids, t, stats, g, tau))


CASES = [
    # R, H, V, K (0: target tokens), dtype, tau
    (1, 8, 1, 0, "bf16", 1.0), (1, 8, 1, 1, "f32", 2.0), (2, 16, 3, 0, "f32", 1.0),
    (3, 8, 5, 4, "bf16", 0.5), (16, 64, 257, 0, "bf16", 1.0), (17, 72, 255, 16, "f32", 1.5),
    (33, 120, 1021, 7, "bf16", 1.0), (40, 256, 1024, 0, "bf16", 1.0), (64, 264, 600, 64, "bf16", 2.0),
    (65, 136, 777, 0, "f32", 1.0), (100, 1016, 513, 5, "bf16", 1.0), (129, 200, 2049, 0, "bf16", 1.0),
    (200, 80, 1500, 33, "f32", 4.0), (257, 328, 1111, 0, "bf16", 1.0), (300, 512, 300, 2, "f32", 1.0),
    (513, 24, 4099, 0, "f32", 1.0), (700, 64, 515, 8, "bf16", 0.75), (1, 4096, 5003, 0, "bf16", 1.0),
    (16, 4096, 4001, 16, "bf16", 1.0), (7, 5376, 2000, 3, "bf16", 1.0), (2, 1032, 20011, 0, "f32", 1.0),
    (12, 64, 70001, 9, "bf16", 1.0), (1030, 136, 1030, 0, "bf16", 1.0),
]


@pytest.mark.parametrize("R,H,V,K,dt,tau", CASES)
def test_sizes(d2, R, H, V, K, dt, tau):
    log(f"lmhead loss R={R} H={H} V={V} K={K} {dt} tau={tau}")
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    x = inputs(R, H, V, K, dtype, R * 7 + V)
    ref = reference(*x, tau)
    loss, gh, gw = run(d2, *x, tau)
    check(ref, loss, gh, gw, dtype, tau)
    # each gradient alone is the same
    h, W, ids, t, g = x
    stats = forward(d2, h, W, ids, t, tau)[1]
    only_h, none = backward(d2, h, W, ids, t, stats, g, tau, need_weight=False)
    assert none is None and torch.equal(only_h, gh)
    none, only_w = backward(d2, h, W, ids, t, stats, g, tau, need_hidden=False)
    assert none is None and torch.equal(only_w, gw)


@pytest.mark.parametrize("R,H,V,dt", [(1024, 16, 70003, "bf16"), (513, 16, 70003, "f32"),
                                      (3000, 8, 25001, "bf16")])
def test_pieces(d2, R, H, V, dt):
    """More than one piece of the vocabulary."""
    log(f"lmhead loss pieces R={R} H={H} V={V} {dt}")
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    x = inputs(R, H, V, 5, dtype, 3)
    x[2][:, 0] = V - 1 - torch.arange(R, device=DEV).int()
    ref = reference(*x, 1.0)
    check(ref, *run(d2, *x, 1.0), dtype, 1.0)


# each way through the kernels, at its ends: rows read whole (up to 16 and 32 rows, by H), rings of 32, 64
# and 128 rows, the weight gradient from held rows (up to 256), streams, rings for the logits of up to 128
# tiles
EDGES = [(R, H, V) for R, V in ((15, 2053), (16, 300), (17, 1031), (32, 4099), (33, 700), (64, 1500),
                                (65, 513), (128, 2049), (129, 1025), (256, 777), (257, 1300))
         for H in (128, 520, 1000, 2056)] + \
    [(16, 3000, 5000), (31, 4096, 3001), (9, 4104, 2003), (48, 4096, 3001), (130, 4096, 1700),
     (600, 2048, 2500), (300, 1544, 40001), (256, 64, 32768), (256, 64, 32769), (512, 72, 16384),
     (512, 72, 16385), (1000, 136, 8191), (1000, 136, 8200), (2000, 64, 4000), (5000, 64, 1500),
     (129, 64, 33001), (256, 72, 40000), (513, 200, 20000), (1300, 136, 9000), (2000, 264, 4500)]


@pytest.mark.parametrize("R,H,V", EDGES)
def test_edges(d2, R, H, V):
    log(f"lmhead loss edges R={R} H={H} V={V}")
    x = inputs(R, H, V, 0 if (R + H) % 2 else 3, torch.bfloat16, R + H)
    x[2][R // 2] = -1
    ref = reference(*x, 1.0)
    check(ref, *run(d2, *x, 1.0), torch.bfloat16, 1.0)


@pytest.mark.parametrize("R", [65, 80, 81, 96, 97, 112, 113, 128, 129, 160, 225, 270, 331])
def test_f32_row_tiles(d2, R):
    log(f"lmhead loss f32 R={R}")
    x = inputs(R, 264, 1203, 0 if R % 2 else 4, torch.float32, R)
    x[2][R // 3] = -1
    check(reference(*x, 1.0), *run(d2, *x, 1.0), torch.float32, 1.0)


@pytest.mark.parametrize("K", [16, 17, 32, 33, 64])
@pytest.mark.parametrize("R,H", [(30, 264), (50, 264), (14, 1200), (25, 1200)])
def test_entries_a_ring_lists(d2, R, H, K):
    """As many entries as the workgroups of few rows look after by themselves, and one more; all of a row's
    in one range of the vocabulary."""
    log(f"lmhead loss R={R} H={H} K={K}")
    V = 20011
    x = inputs(R, H, V, K, torch.bfloat16, R + K)
    x[2][::3] = 5000 + torch.arange(K, device=DEV).int()
    x[2][R - 1] = -1
    ref = reference(*x, 1.0)
    check(ref, *run(d2, *x, 1.0), torch.bfloat16, 1.0)


@pytest.mark.parametrize("R,H,V,dt", [(3, 8, 2200001, "bf16"), (20, 8, 1100003, "bf16"),
                                      (40, 8, 1100003, "bf16"), (2, 8, 1100003, "f32")])
def test_long_vocabulary(d2, R, H, V, dt):
    """More columns than a piece may have."""
    log(f"lmhead loss long vocabulary R={R} V={V} {dt}")
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    x = inputs(R, H, V, 4, dtype, 17)
    x[2][:, 0] = V - 1
    x[2][:, 1] = (1 << 20) - 1
    x[2][:, 2] = 1 << 20
    ref = reference(*x, 1.0)
    check(ref, *run(d2, *x, 1.0), dtype, 1.0)


@pytest.mark.parametrize("R,H", [(3, 8), (40, 8), (3, 1032)])
def test_longest_ranges(d2, R, H):
    """A workgroup's range of the vocabulary is past 2^16 columns: the entries' logits are exact there."""
    log(f"lmhead loss, long ranges R={R} H={H}")
    V = 2 ** 24 + 70001
    gen = torch.Generator(device=DEV).manual_seed(51)
    h = (torch.randint(-5, 6, (R, H), generator=gen, device=DEV) / 4).bfloat16()
    at = torch.tensor([0, 65534, 65535, 65536, 65790, 2 ** 23 + 9, 2 ** 24 + 1, V - 2, V - 1], device=DEV)
    W = torch.zeros(V, H, dtype=torch.bfloat16, device=DEV)
    W[at] = (torch.randint(-2, 3, (at.numel(), H), generator=gen, device=DEV) / 8).bfloat16()
    ids = at.int().expand(R, -1).contiguous()
    t = torch.zeros(R, at.numel(), device=DEV)
    loss, stats = d2.lmhead_distill(h, W, ids, t)
    x = torch.mm(h.double(), W[at].double().t())
    assert torch.equal(stats[:, 2:].double(), x)
    assert torch.equal(stats[:, 0].double(), x.amax(dim=1).clamp(min=0))
    lse = (x.exp().sum(dim=1) + (V - at.numel())).log()
    want = (lse[:, None] - x).mean(dim=1) - math.log(at.numel())
    assert bool(((loss - want).abs() <= eps(V)[0] + U * want.abs()).all())


WAYS = [(14, 1000, 700), (20, 64, 700), (90, 72, 1030), (400, 136, 515), (14, 1200, 700), (25, 1200, 700),
        (400, 136, 20001)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("R,H,V", WAYS)
def test_rows_left_out(d2, R, H, V, dt):
    """Rows without a target: what stands in them, NaN among it, is not read."""
    log(f"lmhead loss rows left out R={R} {dt}")
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    nan, inf = math.nan, math.inf
    for K in (0, 6):
        h, W, ids, t, g = inputs(R, H, V, K, dtype, 5)
        out = torch.zeros(R, dtype=torch.bool, device=DEV)
        out[::3] = True
        out[5:11] = True
        out[R - 1] = True
        h[out] = nan
        h[9] = inf
        g[out] = nan
        first = ids if K == 0 else ids[:, 0]
        if K == 0:
            ids[out] = torch.tensor([-1, V, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32,
                                    device=DEV).repeat(R)[:int(out.sum())]
        else:
            ids[out] = -1
            ids[6] = 3
            t[6] = -inf          # entries without mass
            ids[7], t[7] = V, 4.0
        first[1] = V - 1
        ref = reference(h, W, ids, t, torch.where(out, 0.0, g), 1.0)
        assert int(ref["active"].sum()) == R - int(out.sum())
        loss, gh, gw = run(d2, h, W, ids, t, g, 1.0)
        check(ref, loss, gh, gw, dtype, 1.0)
        assert bool((loss[out] == 0).all()) and bool((gh[out] == 0).all())
        # none left
        if K == 0:
            ids[:] = -1
        else:
            t[:] = -inf
        loss, gh, gw = run(d2, h, W, ids, t, g, 1.0)
        assert bool((loss == 0).all()) and bool((gh == 0).all()) and bool((gw == 0).all())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("R,H,V", WAYS)
def test_entries(d2, R, H, V, dt):
    """Equal ids, fewer entries, masses of every size, a sure row, rows far from 0."""
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    K, tau, inf = 6, 1.25, math.inf
    h, W, ids, t, g = inputs(R, H, V, K, dtype, 6)
    ids[0] = torch.tensor([9, 9, 4, 9, 4, 8])
    ids[1, 3:] = -1
    ids[2, 0], ids[2, 1] = V, 2 ** 31 - 1
    t[3, 2] = -inf
    t[4, 0] = 300.0
    ids[5] = torch.arange(6) + V - 6
    ids[6] = 0
    t[7] = -3e38
    t[8] = 3e38 / 4
    W[11] = 0
    W[11, :8] = 16.0
    h[10, :8] = 16.0                       # logit 2048: the row is sure of token 11
    ids[10] = torch.tensor([11, 11, 11, -1, -1, -1])
    h[12, :8] = -16.0
    ids[12, 0] = 11
    g[13] = 0.0
    ref = reference(h, W, ids, t, g, tau)
    loss, gh, gw = run(d2, h, W, ids, t, g, tau)
    check(ref, loss, gh, gw, dtype, tau)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("R,H,V", WAYS)
def test_not_a_number(d2, R, H, V, dt):
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    nan, inf = math.nan, math.inf
    h, W, ids, t, g = inputs(R, H, V, 4, dtype, 7)
    h[2, 3] = nan
    h[4, 0] = inf
    t[6, 1] = nan
    t[8, 0] = inf
    bad = [2, 4, 6, 8]
    good = torch.tensor([r for r in range(R) if r not in bad], device=DEV)
    hz, tz = torch.nan_to_num(h, 0.0, 0.0, 0.0), torch.nan_to_num(t, 0.0, 0.0, 0.0)
    ref = reference(hz, W, ids, tz, g, 1.0)
    loss, gh, gw = run(d2, h, W, ids, t, g, 1.0)
    assert bool(torch.isnan(loss[bad]).all())
    assert bool(torch.isnan(gh[bad]).any(dim=1).all())
    check(ref, loss, gh, None, dtype, 1.0, rows=good)
    assert bool(torch.isnan(gw[ids[6].long()]).all())
    # an infinite row of W reaches every row's loss (logits of NaN or infinity)
    h, W, ids, t, g = inputs(R, H, V, 0, dtype, 8)
    W[V - 1] = inf
    loss, stats = d2.lmhead_ce(h, W, ids)
    x = torch.mm(h.double(), W.double().t())[:, V - 1]
    assert bool(torch.isnan(loss[torch.isnan(x) | (x == inf)]).all())


def test_against_given_logits(d2):
    """The distillation loss of the logits themselves, on the same (exact) logits."""
    R, H, V, K, tau = 130, 64, 3001, 16, 1.5
    h, W, ids, t, g = inputs(R, H, V, K, torch.float32, 9)
    z = torch.mm(h.double(), W.double().t()).float()
    loss, stats = d2.lmhead_distill(h, W, ids, t, tau)
    want, want_stats = d2.distill(z, ids, t, tau)
    assert torch.equal(stats[:, 0], want_stats[:, 0])
    assert torch.equal(stats[:, 2:], z.gather(1, ids.long()))
    lim = 2 * tau * tau * eps(V)[0] + 2 * U * want.abs()
    assert bool(((loss - want).abs() <= lim).all())


def test_gradients_against_differences(d2):
    """Central differences of the 64-bit loss, off by O(step^2) of its third derivative (the logits
    move by at most step |W| <= 3 step: below 27 step^2 = 3e-9 for a step of 1e-5) and 1e-15 / step."""
    R, H, V, K, tau = 6, 16, 300, 5, 1.5
    h, W, ids, t, g = inputs(R, H, V, K, torch.float32, 11)
    loss, gh, gw = run(d2, h, W, ids, t, g, tau)
    step = 1e-5

    def total(hh, WW):
        return float((reference(hh, WW, ids, t, g, tau)["loss"] * g.double()).sum())

    sigma, eps_q, eps_p = eps(V)
    lim_h = float(g.abs().max()) * tau * (eps_q + eps_p + (V + 64) * 2.0 ** -22) * 6 + 1e-7
    lim_w = float(g.abs().sum()) * tau * (eps_q + eps_p + R * 2.0 ** -22) * 1.25 + 1e-7
    for r, k in ((0, 0), (3, 7), (5, 15)):
        up, dn = h.double(), h.double()
        up[r, k] += step
        dn[r, k] -= step
        d = (total(up, W) - total(dn, W)) / (2 * step)
        assert abs(float(gh[r, k]) - d) <= lim_h
    for v, k in ((0, 0), (int(ids[1, 0]), 5), (int(ids[4, 3]), 9), (V - 1, 15)):
        up, dn = W.double(), W.double()
        up[v, k] += step
        dn[v, k] -= step
        d = (total(h, up) - total(h, dn)) / (2 * step)
        assert abs(float(gw[v, k]) - d) <= lim_w


@pytest.mark.parametrize("K", [0, 9])
def test_autograd(d2, K):
    R, H, V = 50, 64, 1500
    tau = 1.0 if K == 0 else 2.0
    h, W, ids, t, _ = inputs(R, H, V, K, torch.bfloat16, 13)
    w = torch.rand(R, device=DEV)

    def loss_of(hr, Wr):
        return d2.lmhead_ce_loss(hr, Wr, ids) if K == 0 else \
            d2.lmhead_distill_loss(hr, Wr, ids, t, tau)

    hr, Wr = h.clone().requires_grad_(), W.clone().requires_grad_()
    loss = loss_of(hr, Wr)
    (loss * w).sum().backward()
    check(reference(h, W, ids, t, w, tau), loss.detach(), hr.grad, Wr.grad, torch.bfloat16, tau)
    # a frozen head; an expanded gradient
    hr = h.clone().requires_grad_()
    loss = loss_of(hr, W)
    loss.mean().backward()
    m = torch.full((R,), 1.0 / R, device=DEV)
    check(reference(h, W, ids, t, m, tau), loss.detach(), hr.grad, None, torch.bfloat16, tau)
    Wr = W.clone().requires_grad_()
    loss_of(h, Wr)[1:].sum().backward()
    m = torch.ones(R, device=DEV)
    m[0] = 0
    check(reference(h, W, ids, t, m, tau), loss.detach(), None, Wr.grad, torch.bfloat16, tau)
    with torch.no_grad():
        assert not loss_of(hr, Wr).requires_grad


@pytest.mark.parametrize("R,H,V", WAYS)
def test_graph_replay(d2, R, H, V):
    log(f"lmhead loss graph R={R}")
    a, b = inputs(R, H, V, 4, torch.bfloat16, 21), inputs(R, H, V, 4, torch.bfloat16, 22)
    b[2][::2] = -1
    buf = [x.clone() for x in a]
    run(d2, *buf, 1.0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(d2, *buf, 1.0)
    for src in (a, b, a, b):
        for x, y in zip(buf, src):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        want = run(d2, *src, 1.0)
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)


def test_streams_and_slices(d2):
    """Two calls at once on two streams; row vectors that start anywhere; the same bits again."""
    a, b = inputs(300, 264, 5003, 0, torch.bfloat16, 31), inputs(70, 72, 2001, 5, torch.float32, 32)
    wa, wb = run(d2, *a, 1.0), run(d2, *b, 1.0)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s1):
            ga = run(d2, *a, 1.0)
        with torch.cuda.stream(s2):
            gb = run(d2, *b, 1.0)
        torch.cuda.synchronize()
        for got, want in ((ga, wa), (gb, wb)):
            assert all(torch.equal(x, y) for x, y in zip(got, want))
    h, W, ids, _, g = a
    far = torch.cat([ids[:1], ids])[1:], torch.cat([g[:1], g])[1:]
    assert far[0].data_ptr() % 16 != 0
    got = run(d2, h, W, far[0], None, far[1], 1.0)
    assert all(torch.equal(x, y) for x, y in zip(got, wa))


def test_large_head(d2):
    """A head and a gradient past 4 GiB: rows at both ends and past 2^31 and 2^32 bytes."""
    log("lmhead loss, large head")
    R, H, V = 5, 8200, 270001
    gen = torch.Generator(device=DEV).manual_seed(41)
    h = (torch.randint(-5, 6, (R, H), generator=gen, device=DEV) / 4).bfloat16()
    W = torch.zeros(V, H, dtype=torch.bfloat16, device=DEV)
    at = torch.tensor([0, 130000, 130945, 262000, V - 1], device=DEV)
    W[at] = (torch.randint(-1, 2, (5, H), generator=gen, device=DEV) / 8).bfloat16()
    ids = at.int()
    g = torch.randn(R, generator=gen, device=DEV)
    loss, gh, gw = run(d2, h, W, ids, None, g, 1.0)
    x = torch.zeros(R, V, dtype=torch.float64, device=DEV)
    x[:, at] = torch.mm(h.double(), W[at].double().t())
    q = torch.softmax(x, dim=1)
    want = torch.logsumexp(x, dim=1) - x.gather(1, at[:, None])[:, 0]
    sigma, eps_q, eps_p = eps(V)
    assert bool(((loss - want).abs() <= sigma + U * want.abs()).all())
    one = torch.zeros_like(q).scatter_(1, at[:, None], 1.0)
    ag = g.double().abs()[:, None]
    G, hf = (q - one) * g.double()[:, None], 2.0 ** -8
    dG = ag * (q * eps_q + one * eps_p + 1e-30) * (1 + hf) + hf * G.abs()
    aG = G.abs() + dG
    rows = torch.cat([at, torch.tensor([1, 129999, 262143, 262144, V - 2], device=DEV)])
    ah = h.double().abs()
    want = torch.mm(G[:, rows].t(), h.double())
    tol = torch.mm((dG + R * 2.0 ** -23 * aG)[:, rows].t(), ah) * (1 + hf) + hf * want.abs() + 1e-37
    assert bool(((gw[rows].double() - want).abs() <= tol).all())
    want = torch.mm(G[:, at], W[at].double())
    tol = torch.mm((dG + (V + 64) * 2.0 ** -23 * aG)[:, at], W[at].double().abs()) * (1 + hf) + \
        hf * want.abs() + 1e-37
    assert bool(((gh.double() - want).abs() <= tol).all())


def test_most_rows(d2):
    log("lmhead loss, most rows")
    R, H, V = 1 << 16, 8, 300
    x = inputs(R, H, V, 2, torch.bfloat16, 43)
    x[2][torch.arange(R, device=DEV) % 5 == 0] = -1
    ref = reference(*x, 1.0)
    check(ref, *run(d2, *x, 1.0), torch.bfloat16, 1.0)


def test_a_training_step(d2):
    """What a drafter's step calls one after the other: the teacher's side from the top-k pass over
    the target's logits, the loss and its gradients from the hidden states, the norm, the clip."""
    R, H, V, K = 96, 128, 4099, 16
    h, W, _, _, _ = inputs(R, H, V, K, torch.bfloat16, 51)
    teacher_h = inputs(R, H, V, K, torch.bfloat16, 52)[0]
    logits = torch.mm(teacher_h.float(), W.float().t())
    ids, unary, _ = d2.topk_lse(logits, K)
    hr, Wr = h.clone().requires_grad_(), W.clone().requires_grad_()
    loss = d2.lmhead_distill_loss(hr, Wr, ids, unary)
    loss.mean().backward()
    m = torch.full((R,), 1.0 / R, device=DEV)
    ref = reference(h, W, ids, unary, m, 1.0)
    check(ref, loss.detach(), hr.grad, Wr.grad, torch.bfloat16, 1.0)
    grads = [hr.grad, Wr.grad]
    whole = math.sqrt(sum(float((x.double() ** 2).sum()) for x in grads))
    want = [x.double() * min(1.0, 0.25 * whole / whole) for x in grads]
    norm = d2.clip_grads(grads, 0.25 * whole)
    assert abs(float(norm) - whole) <= 4 * U * whole
    for x, y in zip(grads, want):
        assert bool(((x.double() - y).abs() <= (2.0 ** -8 + 8 * U) * y.abs() + 1e-37).all())


@pytest.mark.parametrize("R", [5, 100, 331])
def test_f32_rows_sum_to_zero(d2, R):
    """sum_v G[r][v] is 0 whatever the logits' own rounding: the entry's part is taken from the logit that
    is in the row's sum. Logits of about 1000 that differ by a few (an error of 1e-4 each); grad_hidden's
    first column is the sum, W's first being 1. With u = 2^-24: an exponential errs by 4 u, forward's
    pairs are joined at most 12 times with 7 u each, g / sum, the products and the subtraction by 5 u,
    the sum of 16 terms (whose magnitudes add up to 2) by 32 u, twice that if it truncates:
    4 + 4 + 84 + 5 + 64 < 192."""
    log(f"lmhead loss rows sum to zero R={R}")
    H, V = 2048, 16
    gen = torch.Generator(device=DEV).manual_seed(R)
    h = torch.randn(R, H, generator=gen, device=DEV)
    base = torch.randn(H, generator=gen, device=DEV)
    W = base + torch.randn(V, H, generator=gen, device=DEV) * 0.05
    h = h * 0.3 + base * 0.5
    h[:, 0], W[:, 0] = 0.0, 1.0
    ids = torch.mm(h, W.t()).argmax(dim=1).int()
    g = torch.ones(R, device=DEV)
    loss, stats = d2.lmhead_ce(h, W, ids)
    gh, _ = d2.lmhead_ce_backward(h, W, ids, stats, g, need_weight=False)
    assert float(stats[:, 0].min()) > 500.0
    assert float(gh[:, 0].abs().max()) <= 192 * U


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("R,H,V", [(12, 1200, 700), (25, 1200, 700), (30, 264, 700), (60, 264, 700),
                                   (100, 264, 700), (200, 264, 700), (300, 264, 700)])
def test_large_scale(d2, R, H, V, dt):
    """g tau passes the largest fp32 number, the gradient does not: with K equal entries |G| < g tau / K
    at an entry and g tau q elsewhere, and q is about 1 / V where tau is large. (Six rows of that scale: their
    sums, at most 6 g tau / 16 * 5 / 4, are finite too.)"""
    log(f"lmhead loss, large scale R={R} H={H} V={V} {dt}")
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    for K, tau, size in ((64, 1e20, 4e18), (16, 1e20, 4e18), (64, 1e38, 4.0), (16, 1e-20, 1e-10)):
        tau = float(torch.tensor(tau, dtype=torch.float32))  # (it is passed in fp32)
        h, W, ids, t, g = inputs(R, H, V, K, dtype, R + K)
        t.zero_()
        ids[:] = torch.arange(K, device=DEV)
        ids[4] = -1
        g = torch.where(g > 0, 1.0, -1.0) * size
        g[6:] *= 1e-3
        ref = reference(h, W, ids, t, g, tau)
        loss, stats = forward(d2, h, W, ids, t, tau)
        gh, gw = backward(d2, h, W, ids, t, stats, g, tau)
        assert bool(torch.isfinite(gh).all()) and bool(torch.isfinite(gw).all())
        loss.zero_()  # (tau^2 may pass the largest number in it, and it is not what is tested)
        ref["loss"].zero_()
        check(ref, loss, gh, gw, dtype, tau)


WORKSPACES = [(3, 64, 700), (14, 1200, 900), (25, 1200, 900), (30, 264, 1000), (50, 264, 1000), (100, 72, 1030),
              (140, 136, 515), (250, 136, 515), (600, 264, 3000), (300, 64, 20000), (140, 72, 34000)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("R,H,V", WORKSPACES)
def test_workspace_as_it_comes(d2, monkeypatch, R, H, V, dt):
    """Nothing is taken from a workspace that the call has not written: it starts as NaN. All rows, a
    few, one, none."""
    log(f"lmhead loss workspace R={R} H={H} V={V} {dt}")
    monkeypatch.setattr(d2, "_workspace", lambda n, device: torch.full((max(int(n), 16),), 255,
                                                                       dtype=torch.uint8, device=device))
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    for K, step in ((0, 1), (3, 1), (0, 7), (20, 7), (0, R + 1), (2, R + 1), (0, 0)):
        x = inputs(R, H, V, K, dtype, R + step)
        if step != 1:
            out = torch.ones(R, dtype=torch.bool, device=DEV)
            if step:
                out[R // 2::step] = False
            x[2][out] = -1
        check(reference(*x, 1.0), *run(d2, *x, 1.0), dtype, 1.0)
