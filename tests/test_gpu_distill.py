"""Distillation from a teacher's top logits vs a plain implementation in 64 bits (needs an MI355X).

Tolerances, with u = 2^-24 (half a step of fp32, relative) and the row's largest logit m:
  * Sigma = sum exp((z - m) / tau): a term's exponent t = (z - m) log2(e) / tau errs by the rounding
    of the fma and of log2(e) / tau, at most 2 |t| u, which is 2 |t| u ln 2 of the term; terms with
    |t| > 64 add up to less than V 2^-64 and do not count; the hardware exponential errs by one
    step (2 u). The sum is a chain of at most kChain additions per thread and a tree of at most
    16 joins (a rescale, rounded exponential and sum each: 4 u). So Sigma errs by at most
      eps_sigma = (2 * 64 * ln 2 + 2 + kChain + 64) u    of itself.
  * loss: everything after Sigma is fp64: tau^2 eps_sigma (the p_j add up to 1), and the final
    rounding, u |loss|.
  * gradient: q has the same exponent error again, the rounding of Sigma and of the coefficient and
    the products: eps_q = eps_sigma + (2 * 64 * ln 2 + 2 + 4) u; so |g| tau q eps_q, and the final
    rounding: u |ref| in fp32, 2^-8 |ref| in bf16. q < 2^-100 may be flushed: + 1e-30 |g| tau.
kChain: a thread adds at most ceil(V / 512) + 16 terms in a slice (fewer per accumulator).
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


def reference(z, ids, t, g, tau):
    """Loss, gradient and q in 64 bits on the host, from the formulas."""
    z, t, g = z.cpu().double(), t.cpu().double(), g.cpu().double()
    ids = ids.cpu().long()
    R, V = z.shape
    loss, grad, q = torch.zeros(R).double(), torch.zeros(R, V).double(), torch.zeros(R, V).double()
    for r in range(R):
        ok = (ids[r] >= 0) & (ids[r] < V)
        i, a = ids[r][ok], t[r][ok] / tau
        if len(i) == 0 or bool((a == -math.inf).all()):
            continue
        p = torch.exp(a - a.max())
        p = p / p.sum()
        if bool((z[r] == -math.inf).all()):
            loss[r] = math.inf
            continue
        log_q = (z[r] - z[r].max()) / tau
        log_q = log_q - torch.log(torch.exp(log_q).sum())
        q[r] = torch.exp(log_q)
        terms = torch.where(p == 0, 0.0, p * (torch.log(p) - log_q[i]))
        loss[r] = tau * tau * terms.sum()
        d = q[r].clone()
        d.index_add_(0, i, -p)
        grad[r] = g[r] * tau * d
    return loss, grad, q


def eps_sigma(V):
    chain = -(-V // 512) + 16
    return (2 * 64 * math.log(2) + 2 + chain + 64) * U


def check(got_loss, got_grad, ref, V, tau, g, dtype):
    loss, grad, q = ref
    if got_loss is not None:
        got = got_loss.cpu().double()
        assert torch.equal(torch.isnan(got), torch.isnan(loss))
        assert torch.equal(torch.isinf(got), torch.isinf(loss))
        f = torch.isfinite(loss)
        tol = tau * tau * eps_sigma(V) + U * loss[f].abs()
        assert bool(((got[f] - loss[f]).abs() <= tol).all()), (got[f] - loss[f]).abs().max()
    if got_grad is not None:
        got = got_grad.cpu().double()
        assert torch.equal(torch.isnan(got), torch.isnan(grad))
        half = U if dtype == torch.float32 else 2.0 ** -8
        eps_q = eps_sigma(V) + (2 * 64 * math.log(2) + 6) * U
        ag = g.cpu().double().abs()[:, None] * tau
        tol = (ag * q * eps_q) * (1 + half) + half * grad.abs() + 1e-30 * ag
        err = (got - grad).abs()
        bad = ~torch.isnan(grad) & ~(err <= tol)
        assert not bool(bad.any()), (bad.nonzero()[:4], got[bad][:4], grad[bad][:4])


def inputs(R, V, K, dtype, seed, spread=3.0):
    gen = torch.Generator().manual_seed(seed)
    z = (torch.randn(R, V, generator=gen) * spread).to(dtype)
    ids = torch.stack([torch.randperm(V, generator=gen)[:K] if V < 5000 else
                       torch.randint(0, V // K, (K,), generator=gen) + torch.arange(K) * (V // K)
                       for _ in range(R)]).int()
    t = torch.randn(R, K, generator=gen) * 2
    g = torch.randn(R, generator=gen)
    return z.to(DEV), ids.to(DEV), t.to(DEV), g.to(DEV)


def run_all(d2, z, ids, t, g, tau):
    """(loss, gradient) of the two calls and of the single one, written into guarded buffers."""
    R, V = z.shape
    loss, stats = d2.distill(z, ids, t, tau)

    def guarded():
        pad = 64
        whole = torch.full((R * V + 2 * pad,), 7.0, dtype=z.dtype, device=DEV)
        return whole, whole[pad:pad + R * V].view(R, V)

    outs = []
    w1, o1 = guarded()
    d2.distill_backward(z, ids, t, stats, g, tau, out=o1)
    w2, o2 = guarded()
    loss2, _ = d2.distill_step(z, ids, t, g, tau, out=o2)
    torch.cuda.synchronize()
    for w in (w1, w2):
        assert bool((w[:64] == 7).all()) and bool((w[64 + R * V:] == 7).all())
    return (loss, o1), (loss2, o2)


CASES = [
    # R, V, K, dtype, tau
    (1, 1, 1, "f32", 1.0), (1, 1, 1, "bf16", 2.0), (3, 2, 2, "bf16", 1.0), (5, 7, 3, "f32", 0.5),
    (4, 9, 9, "bf16", 1.0), (9, 64, 16, "f32", 1.0), (7, 1021, 64, "bf16", 1.5),
    (33, 4099, 5, "f32", 4.0), (1030, 515, 8, "bf16", 1.0), (1025, 1023, 3, "f32", 0.75),
    (2, 32003, 33, "f32", 1.0), (16, 151936, 16, "bf16", 1.0), (3, 262143, 64, "bf16", 2.0),
    (1, 151937, 1, "f32", 1.0), (1024, 8200, 64, "bf16", 0.25), (1024, 16391, 1, "f32", 1.0),
]


@pytest.mark.parametrize("R,V,K,dt,tau", CASES)
def test_sizes(d2, R, V, K, dt, tau):
    log(f"distill R={R} V={V} K={K} {dt} tau={tau}")
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    z, ids, t, g = inputs(R, V, K, dtype, R * 7 + V)
    ref = reference(z, ids, t, g, tau)
    for loss, grad in run_all(d2, z, ids, t, g, tau):
        check(loss, grad, ref, V, tau, g, dtype)


# slices; a row per workgroup forward, slices backward; a row per workgroup; held in registers
WAYS = [(16, 165000), (16, 60000), (1100, 600), (130, 20001)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("R,V", WAYS)
def test_special_rows(d2, R, V, dt):
    log(f"distill special rows R={R} V={V} {dt}")
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    inf, low = math.inf, torch.finfo(dtype).min
    K, tau = 6, 1.25
    z, ids, t, g = inputs(R, V, K, dtype, 5)
    z[0, 100:300] = -inf                   # masked tokens no entry names
    ids[0] = torch.tensor([1, 2, 3, 4, 5, 6])
    ids[1] = -1                            # no entries
    ids[2, 3:] = -1                        # fewer entries
    ids[3] = torch.tensor([9, 9, 4, 9, 4, 8])   # the same id twice and three times
    ids[4, 0], ids[4, 1] = V, 2 ** 31 - 1       # out of range: no entries
    t[5] = -inf                            # entries without mass
    t[6, 2] = -inf
    z[7, 50] = -inf                        # an entry at a masked token
    ids[7, 1] = 50
    z[8] = -inf                            # nothing left of the student's row
    z[9] = low                             # a row of the type's lowest value
    z[10, :V // 2] = low                   # half of it masked that way
    ids[10] = torch.arange(6) + V // 2
    z[11] = -inf                           # one token left
    z[11, 17] = 3.0
    ids[11, :] = -1
    ids[11, 0] = 17
    z[12] = z[12].abs() * 1e37             # far above: differences decide
    z[13] = 30000.0
    ids[14, 0] = V - 1                     # the row's ends
    ids[14, 1] = 0
    ref = reference(z, ids, t, g, tau)
    for loss, grad in run_all(d2, z, ids, t, g, tau):
        check(loss, grad, ref, V, tau, g, dtype)
        assert bool((grad[1] == 0).all()) and float(loss[1]) == 0.0
        assert bool((grad[5] == 0).all()) and float(loss[5]) == 0.0
        assert float(loss[8]) == inf and bool((grad[8] == 0).all())
        assert float(loss[7]) == inf


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("R,V", WAYS)
def test_not_a_number(d2, R, V, dt):
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    z, ids, t, g = inputs(R, V, 4, dtype, 6)
    z[2, 5] = math.nan
    z[4, V - 1] = math.inf
    t[6, 1] = math.nan
    z[8] = -math.inf
    z[8, 3] = math.nan
    ids[9] = -1
    z[9, 7] = math.nan                     # without entries the row stays out of it
    bad = [2, 4, 6, 8]
    good = [r for r in range(R) if r not in bad]
    ref = reference(z, ids, t, g, 1.0)
    for loss, grad in run_all(d2, z, ids, t, g, 1.0):
        assert bool(torch.isnan(loss[bad]).all())
        assert bool(torch.isnan(grad[[2, 4, 8]]).any(dim=1).all())
        assert bool(torch.isnan(grad[6][ids[6].long()]).all())
        check(loss[good], grad[good], tuple(x[good] for x in ref), V, 1.0, g[good], dtype)


@pytest.mark.parametrize("V,dt", [(40000, "bf16"), (70011, "bf16"), (140001, "bf16"),
                                  (180003, "bf16"), (20003, "f32"), (40001, "f32"), (66666, "f32"),
                                  (90007, "f32")])
def test_long_rows(d2, V, dt):
    """Many long rows (held in registers between the passes, wholly or in part): a few rows of each
    kind against the formulas, the others against the two calls."""
    log(f"distill long rows V={V} {dt}")
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    R, K, tau = 1024, 9, 1.5
    gen = torch.Generator(device=DEV).manual_seed(V)
    z = (torch.randn(R, V, generator=gen, device=DEV) * 3).to(dtype)
    ids = (torch.arange(K, device=DEV) * (V // K) +
           torch.randint(0, V // K, (R, K), generator=gen, device=DEV)).int()
    t = torch.randn(R, K, generator=gen, device=DEV)
    g = torch.rand(R, generator=gen, device=DEV) - 0.5
    inf, low = math.inf, torch.finfo(dtype).min
    ids[1] = -1
    ids[2, 4:] = ids[2, 0]
    z[3, V // 3:] = -inf
    z[4] = -inf
    z[5] = low
    z[6, :V // 2] = low
    z[7] = z[7].abs() * 1e37
    z[8, V - 2] = math.nan
    z[9, 1] = inf
    z[10] = -inf
    z[10, V // 2] = math.nan
    ids[11, 0], ids[11, 1] = 0, V - 1
    z[12] = z[12] * 1e7                    # no reference, but no mask either
    loss, grad = d2.distill_step(z, ids, t, g, tau)
    rows = [0, 1, 2, 3, 4, 5, 6, 7, 11, 12, 511, 1023]
    ref = reference(z[rows], ids[rows], t[rows], g[rows], tau)
    check(loss[rows], grad[rows], ref, V, tau, g[rows], dtype)
    bad = [8, 9, 10]
    assert bool(torch.isnan(loss[bad]).all()) and bool(torch.isnan(grad[bad]).any(dim=1).all())
    two, stats = d2.distill(z, ids, t, tau)
    grad2 = d2.distill_backward(z, ids, t, stats, g, tau)
    good = [r for r in range(R) if r not in bad]
    fin = torch.isfinite(two)
    assert torch.equal(fin, torch.isfinite(loss))
    tol = 2 * (tau * tau * eps_sigma(V) + U * two[fin].abs())
    assert bool(((loss[fin] - two[fin]).abs() <= tol).all())
    half = U if dt == "f32" else 2.0 ** -8
    # both sides within their tolerance of the formula: |q - p| <= 1, q <= 1
    lim = 2 * (g.abs() * tau)[:, None] * (eps_sigma(V) + 200 * U) + \
        2 * half * torch.maximum(grad.float().abs(), grad2.float().abs())
    assert bool(((grad.float() - grad2.float()).abs() <= lim)[good].all())


def test_gradient_against_differences(d2):
    """Central differences of the 64-bit loss at a step of 1e-5: off by O(h^2) = 1e-10 of the third
    derivative (below tau^-1) and 1e-16 / h of the loss."""
    R, V, K, tau = 4, 2053, 7, 1.5
    z, ids, t, g = inputs(R, V, K, torch.float32, 11)
    loss, grad = d2.distill_step(z, ids, t, g, tau)
    h = 1e-5
    z64 = z.cpu().double()
    one = torch.ones(R)
    for r in range(R):
        for v in [0, V - 1, 512] + ids[r, :3].tolist():
            up, dn = z64.clone(), z64.clone()
            up[r, v] += h
            dn[r, v] -= h
            d = (reference(up, ids, t, one, tau)[0][r] - reference(dn, ids, t, one, tau)[0][r])
            want = float(d / (2 * h)) * float(g[r])
            q_tol = abs(float(g[r])) * tau * (eps_sigma(V) + 100 * U)
            assert abs(float(grad[r, v]) - want) <= q_tol + 1e-8, (r, v)


def test_autograd(d2):
    R, V, K, tau = 12, 3001, 9, 2.0
    z, ids, t, _ = inputs(R, V, K, torch.bfloat16, 3)
    w = torch.rand(R, device=DEV)
    zr = z.clone().requires_grad_()
    loss = d2.distill_loss(zr, ids, t, tau)
    (loss * w).sum().backward()
    ref = reference(z, ids, t, w, tau)
    check(loss.detach(), zr.grad, ref, V, tau, w, torch.bfloat16)
    # a part of the rows (a gradient that is a view), and an expanded one
    zr.grad = None
    d2.distill_loss(zr, ids, t, tau)[1:].sum().backward()
    w1 = torch.ones(R, device=DEV)
    w1[0] = 0
    check(None, zr.grad, reference(z, ids, t, w1, tau), V, tau, w1, torch.bfloat16)
    # through the product that makes the logits
    h = torch.randn(R, 64, device=DEV, requires_grad=True)
    W = torch.randn(V, 64, device=DEV, requires_grad=True)
    d2.distill_loss(h @ W.t(), ids, t, tau).mean().backward()
    assert bool(torch.isfinite(h.grad).all()) and bool(torch.isfinite(W.grad).all())


def test_most_rows(d2):
    log("distill, most rows")
    R, V, K = 1 << 21, 3, 2
    gen = torch.Generator(device=DEV).manual_seed(19)
    z = torch.randn(R, V, generator=gen, device=DEV)
    ids = torch.randint(-1, V, (R, K), generator=gen, device=DEV, dtype=torch.int32)
    t = torch.randn(R, K, generator=gen, device=DEV)
    g = torch.rand(R, generator=gen, device=DEV)
    q = torch.softmax(z.double(), 1)
    has = ids >= 0
    p = torch.softmax(t.double().masked_fill(~has, -math.inf), 1).nan_to_num(0.0)
    ln = torch.where(has, torch.log(p) - torch.log(q).gather(1, ids.clamp(min=0).long()), 0.0)
    want = (p * ln).sum(1)
    grad = q.clone().scatter_add_(1, ids.clamp(min=0).long(), torch.where(has, -p, 0.0))
    grad = torch.where(has.any(1, keepdim=True), grad, 0.0) * g[:, None].double()
    for loss, got in ((d2.distill_step(z, ids, t, g)),
                      (d2.distill(z, ids, t)[0],
                       d2.distill_backward(z, ids, t, d2.distill(z, ids, t)[1], g))):
        assert bool(((loss.double() - want).abs() <= eps_sigma(V) + U * want.abs()).all())
        lim = g[:, None].double() * (eps_sigma(V) + 200 * U) + U * grad.abs()
        assert bool(((got.double() - grad).abs() <= lim).all())


def test_no_gradient_needed(d2):
    z, ids, t, _ = inputs(3, 100, 4, torch.float32, 3)
    with torch.no_grad():
        assert not d2.distill_loss(z, ids, t).requires_grad


@pytest.mark.parametrize("R,V", WAYS)
def test_graph_replay(d2, R, V):
    log(f"distill graph R={R} V={V}")
    z, ids, t, g = inputs(R, V, 8, torch.bfloat16, 21)
    z2, ids2, t2, g2 = inputs(R, V, 8, torch.bfloat16, 22)
    buf = [x.clone() for x in (z, ids, t, g)]
    graph = torch.cuda.CUDAGraph()
    d2.distill_step(*buf)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        loss, stats = d2.distill(*buf[:3])
        grad = d2.distill_backward(*buf[:3], stats, buf[3])
        loss_s, grad_s = d2.distill_step(*buf)
    for src in ((z, ids, t, g), (z2, ids2, t2, g2), (z, ids, t, g)):
        for b, x in zip(buf, src):
            b.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        want, st = d2.distill(*src[:3])
        want_g = d2.distill_backward(*src[:3], st, src[3])
        want_s = d2.distill_step(*src)
        torch.cuda.synchronize()
        assert torch.equal(loss, want) and torch.equal(grad, want_g)
        assert torch.equal(loss_s, want_s[0]) and torch.equal(grad_s, want_s[1])


def test_other_stream_and_two_at_once(d2):
    a = inputs(16, 165000, 8, torch.bfloat16, 31)
    b = inputs(700, 3001, 8, torch.float32, 32)
    wa, wb = d2.distill_step(*a), d2.distill_step(*b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s1):
            ga = d2.distill_step(*a)
        with torch.cuda.stream(s2):
            gb = d2.distill_step(*b)
        torch.cuda.synchronize()
        for got, want in ((ga, wa), (gb, wb)):
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_teacher_from_the_top_k_pass(d2):
    """The teacher's side as topk_lse gives it; a student equal to the teacher, kept whole, has
    loss 0 and gradient 0 up to the tolerances."""
    R, V, K = 20, 5003, 16
    z, _, _, g = inputs(R, V, K, torch.float32, 41)
    ids, unary, _ = d2.topk_lse(z, K)
    ref = reference(z, ids, unary, g, 1.0)
    loss, grad = d2.distill_step(z, ids, unary, g)
    check(loss, grad, ref, V, 1.0, g, torch.float32)
    few = z[:, :K].contiguous()
    ids, unary, _ = d2.topk_lse(few, K)
    loss, grad = d2.distill_step(few, ids, unary, g)
    check(loss, grad, reference(few, ids, unary, g, 1.0), K, 1.0, g, torch.float32)
    assert float(loss.abs().max()) <= 2e-5
