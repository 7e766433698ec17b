"""Sampling from whole rows of logits vs a plain implementation in 64 bits (needs an MI355X).

The reference sorts a row (logit descending, id ascending), sums its weights in 64 bits and applies
the definition. A weight on the GPU errs by at most, relative to itself: half a step of its 41-bit
second factor, which is at least 0.989 (2^-41.98), the polynomial of that factor (2^-42.5; bf16 rows
multiply two of them and have no fixed-point step) and the fp64 roundings of its argument (below 4096,
2^-46): below 2^-41 in all. A running sum errs by no more than that of itself, and its comparison with a
cut (a product with a sum that errs as much, or with two) by less than 2^-38 of the row's mass. So:
  * the token is the reference's, unless a cut or the draw lies within 2^-38 of the mass of a
    running sum, where either neighbour's answer is right; the inputs below have no such place
    (asserted: `clear`), but for runs of equal largest logits, whose sums are whole numbers and exact
    on both sides;
  * logprob errs by 2^-37 (a quotient of sums, its logarithm) and its rounding to fp32, 2^-24 of
    itself.
"""
import math
import sys

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def log(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module")
def d2():
    import dflash2_draft_candidate_amd
    return dflash2_draft_candidate_amd


def f32(x):
    return float(np.float32(x))


def reference_row(x, T, k, p, m, u):
    """(token, logprob, clear): clear says that no cut is within 2^-38 of a running sum."""
    x = np.where(np.isnan(x), -np.inf, x)
    if x.max() == -np.inf:
        return -1, -math.inf, True
    order = np.lexsort((np.arange(len(x)), -x))
    if not T > 0:
        return int(order[0]), 0.0, True
    v = x[order]
    with np.errstate(invalid="ignore"):
        w = np.where(v == v[0], 1.0, np.exp((v - v[0]) / T))
    w[~(w >= 2.0 ** -64)] = 0
    N = int((w > 0).sum())
    w, order = w[:N], order[:N]
    S = np.cumsum(w)
    n = min(k, N) if k >= 1 else N
    Z = S[n - 1]
    clear = True

    def close(target, n):
        i = int(np.searchsorted(S, target))
        near = S[max(i - 1, 0):i + 1]
        exact = bool((w[:max(n, i + 1)] == 1).all())  # whole numbers
        return not exact and bool((np.abs(near - target) <= 2.0 ** -38 * S[-1]).any())
    cuts = [n]
    if p < 1:
        cuts.append(int(np.argmax(S >= p * Z)) + 1)
        clear &= not close(p * Z, n)
    if m > 0:
        cuts.append(int((w >= min(m, 1.0)).sum()))
    n = max(1, min(cuts))
    W = S[n - 1]
    i = int(np.argmax(S[:n] > u * W))
    clear &= not close(u * W, n) or u == 0
    return int(order[i]), float(np.log(w[i] / W)), clear


def check(d2, x, u, T=1.0, k=0, p=1.0, m=0.0, out=None):
    """x [R, V] on the host (fp32 or bf16); settings numbers or lists."""
    R = x.shape[0]
    full = lambda v: list(v) if isinstance(v, (list, np.ndarray)) else [v] * R
    dev = lambda v, dt: torch.tensor(v, dtype=dt, device=DEV) if isinstance(v, (list, np.ndarray)) else v
    ids, lp = d2.sample(x.to(DEV), torch.tensor(u, dtype=torch.float32, device=DEV),
                        dev(T, torch.float32), dev(k, torch.int32), dev(p, torch.float32),
                        dev(m, torch.float32), out=out)
    ids, lp = ids.cpu().tolist(), lp.cpu().double().tolist()
    xs = x.double().numpy()
    Ts, ks, ps, ms = full(T), full(k), full(p), full(m)
    for r in range(R):
        want, wlp, clear = reference_row(xs[r], f32(Ts[r]), ks[r], f32(ps[r]), f32(ms[r]), f32(u[r]))
        assert clear, f"row {r}: the inputs leave the answer open"
        assert ids[r] == want, f"row {r}: token {ids[r]}, expected {want} (T={Ts[r]} k={ks[r]} " \
            f"p={ps[r]} m={ms[r]} u={u[r]})"
        if math.isinf(wlp):
            assert lp[r] == wlp
        else:
            assert abs(lp[r] - wlp) <= 2.0 ** -37 + 2.0 ** -24 * abs(wlp), (r, lp[r], wlp)


def rows(R, V, dt, seed, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(R, V, generator=g) * spread
    boost = torch.randint(0, V, (R, 3), generator=g)
    x.scatter_add_(1, boost, 8 * torch.rand(R, 3, generator=g))
    u = torch.rand(R, generator=g).tolist()
    return x.to(torch.float32 if dt == "f32" else torch.bfloat16), u


SETTINGS = [
    dict(), dict(T=0.7), dict(T=0.0), dict(k=1), dict(k=40), dict(T=1.3, k=300), dict(p=0.9),
    dict(T=0.6, p=0.5), dict(m=0.05), dict(T=1.5, m=0.001), dict(k=50, p=0.95, T=0.8),
    dict(k=900, p=0.99, m=0.01, T=2.0), dict(p=0.0), dict(m=1.0), dict(T=8.0), dict(T=0.01),
]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("R,V", [(1, 1), (3, 2), (2, 7), (5, 9), (4, 100), (6, 1021), (3, 4099),
                                 (2, 50021), (2, 151936), (1, 262143)])
def test_sizes(d2, R, V, dt):
    log(f"sample R={R} V={V} {dt}")
    x, u = rows(R, V, dt, R * 31 + V)
    for i, s in enumerate(SETTINGS):
        check(d2, x, [(v + 0.37 * i) % 1.0 for v in u], **s)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_settings_of_each_row(d2, dt):
    R, V = 48, 6007
    x, u = rows(R, V, dt, 77)
    s = [SETTINGS[i % len(SETTINGS)] for i in range(R)]
    check(d2, x, u, T=[a.get("T", 1.0) for a in s], k=[a.get("k", 0) for a in s],
          p=[a.get("p", 1.0) for a in s], m=[a.get("m", 0.0) for a in s])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("spread", [0.0, 1e-4, 0.02, 0.3, 30.0])
@pytest.mark.parametrize("V", [40000, 80000])  # (bf16: a workgroup per row; slices)
def test_flat_and_steep_rows(d2, V, spread, dt):
    """Many tokens in a bin: bins are split by value, down to a single value in constant rows."""
    log(f"sample spread={spread} {dt}")
    g = torch.Generator().manual_seed(9)
    R = 4
    x = (torch.randn(R, V, generator=g) * spread + 1.5)
    x = x.to(torch.float32 if dt == "f32" else torch.bfloat16)
    for i, s in enumerate([dict(), dict(T=0.5, p=0.7), dict(k=20000), dict(k=1500, p=0.5),
                           dict(T=3.0, m=0.99), dict(k=30000, p=0.9, m=0.5)]):
        check(d2, x, [0.013 + 0.11 * i, 0.5, 0.77, 0.9995], **s)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_ties(d2, dt):
    """Equal logits at every cut go to the lower id; signed zeros are equal."""
    V = 3000
    x = torch.zeros(5, V)
    x[0, 1000:1010] = 4.0
    x[1, ::2] = -0.0
    x[2, 5:2900] = 2.0
    x[3] = 1.0
    x[3, 17] = 2.0
    x[4, ::3] = 0.5
    x = x.to(torch.float32 if dt == "f32" else torch.bfloat16)
    for s in (dict(k=4), dict(k=1), dict(p=0.3), dict(k=2000, p=0.5), dict(), dict(T=0.25, m=0.9)):
        for u in (0.0, 0.21, 0.83, 1.0 - 2.0 ** -24):
            check(d2, x, [u] * 5, **s)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_masks(d2, dt):
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    V, inf, low = 5001, math.inf, torch.finfo(dtype).min
    x, u = rows(12, V, dt, 3)
    x[0] = -inf                     # nothing left
    x[1, 1:] = -inf                 # one token left
    x[2, ::2] = -inf
    x[3] = low                      # all at the type's lowest value
    x[4, 100:] = low
    x[5, :2500] = math.nan
    x[6] = math.nan                 # nothing left either
    x[7, 40] = inf                  # one infinite logit, several, and ties among them
    x[8, 40:60] = inf
    x[9] = inf
    x[10] = torch.finfo(dtype).max
    x[11, V - 1] = 60.0
    for s in SETTINGS:
        check(d2, x, u, **s)
    for v in (0.0, 0.5, 1.0 - 2.0 ** -24):
        check(d2, x, [v] * 12, k=7, p=0.6)


def test_values_outside_the_counted_range(d2):
    """bf16 rows with values below 2^-20 (gathered, or too many) and from 2^8 on, in rows that are
    counted whole and rows that are cut into slices."""
    for V in (6001, 80010):
        x, u = rows(10, V, "bf16", V)
        g = torch.Generator().manual_seed(V)
        tiny = (torch.randn(V, generator=g) * 2.0 ** -22).to(torch.bfloat16)
        at = torch.randperm(V, generator=g)
        x[0, at[:40]] = tiny[:40]                       # a few, between the others
        x[1] = -x[1].abs() - 0.5
        x[1, at[:30]] = tiny[:30]                       # they are the top
        x[2] = -x[2].abs() - 0.5
        x[2, at[:64]] = 0.0                             # as many as are gathered, all equal
        x[3, at[:65]] = -0.0                            # one more
        x[4] = tiny                                     # nothing else
        x[5, at[:7]] = 300.0                            # large
        x[6, at[:700]] = -300.0                         # large negative: no weight, or some
        x[7] = -1000.0 - x[7].abs()
        x[8] = -torch.inf
        x[8, at[:3]] = tiny[:3]
        x[9] = 5e-324
        for i, s in enumerate(SETTINGS + [dict(T=100.0), dict(T=50.0, k=V // 2, p=0.9)]):
            check(d2, x, [(v + 0.29 * i) % 1.0 for v in u], **s)


@pytest.mark.parametrize("R,V", [(256, 300000), (1, 1200000)])
def test_a_value_more_often_than_a_half_word_counts(d2, R, V):
    """Constant rows: a part of the row holds one value more than 65535 times."""
    x = torch.zeros(R, V, dtype=torch.bfloat16, device=DEV)
    x[R - 1] = 1.5
    u = (torch.arange(R, device=DEV) + 0.5) / R
    ids, lp = d2.sample(x, u)
    assert ids.tolist() == [int(v * V) for v in u.double().tolist()]
    assert float((lp.double() + math.log(V)).abs().max()) <= 2.0 ** -37 + 2.0 ** -24 * math.log(V)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_late_maximum(d2, dt):
    """Rows whose first logits say little of their maximum: masked, far below it, just below the bins'
    headroom, or NaN; the bf16 rows hold a large logit, which sends them the same way."""
    V, inf = 40000, math.inf
    x, u = rows(8, V, "f32", 71)
    x[0, :30000] = -inf
    x[1, 39000] = 60.0                 # far above everything
    x[2, 39000:39005] = 45.0
    x[3, :20000] -= 40.0
    x[4, :39999] = -inf
    x[5, :9000] = math.nan
    x[6] = -x[6].abs() * 100           # steep, all negative
    x[7, 20000:] += 25.0
    if dt == "bf16":
        x = x.to(torch.bfloat16)
        x[:, 17] = 300.0
        x[4, 17] = -inf
    else:
        x = x.float()
    for i, s in enumerate([dict(), dict(T=0.5), dict(T=0.05, p=0.9), dict(T=1.4, p=0.97),
                           dict(T=2.0, k=2000, p=0.9), dict(T=3.0, m=0.05), dict(T=20.0, p=0.8),
                           dict(T=40.0, m=0.2, p=0.6), dict(T=0.0)]):
        check(d2, x, [(v + 0.31 * i) % 1.0 for v in u], **s)


@pytest.mark.parametrize("R,V", [(5, 150001), (130, 150001)])  # slices; a workgroup per row
def test_mostly_masked_rows(d2, R, V):
    """Rows of which little is left, as constrained decoding makes them: more masks than a half-word
    counts."""
    x, u = rows(5, V, "bf16", 101)
    g = torch.Generator().manual_seed(102)
    off = torch.rand(5, V, generator=g)
    x[0, off[0] > 0.1] = -math.inf
    x[1, off[1] > 0.001] = torch.finfo(torch.bfloat16).min
    x[2, off[2] > 0.5] = -math.inf
    x[2, off[2] > 0.8] = -300.0
    x[3, :] = -math.inf
    x[3, V - 3] = -2.0
    x[4, off[4] > 0.0005] = math.nan
    x = x.repeat(R // 5, 1)
    for i, s in enumerate([dict(), dict(p=0.9), dict(T=0.7, k=40), dict(T=2.0, m=0.02, p=0.97)]):
        v = [(a + 0.23 * i) % 1.0 for a in u]
        ids, lp = d2.sample(x.to(DEV), torch.tensor(v * (R // 5), device=DEV),
                            s.get("T", 1.0), s.get("k", 0), s.get("p", 1.0), s.get("m", 0.0))
        assert torch.equal(ids, ids[:5].repeat(R // 5)) and torch.equal(lp, lp[:5].repeat(R // 5))
        if R == 5:
            check(d2, x, v, **s)
        else:
            few = d2.sample(x[:5].to(DEV), torch.tensor(v, device=DEV),
                            s.get("T", 1.0), s.get("k", 0), s.get("p", 1.0), s.get("m", 0.0))
            assert torch.equal(ids[:5], few[0])


def test_any_top_k_number(d2):
    x, u = rows(3, 500, "f32", 11)
    x, u = x.to(DEV), torch.tensor(u, device=DEV)
    want = d2.sample(x, u)[0]
    for k in (0, -3, -2 ** 40, 500, 2 ** 40):
        assert torch.equal(d2.sample(x, u, top_k=k)[0], want)


def test_very_long_rows(d2):
    """More groups than their maxima are kept for, in both types."""
    V = 600011
    for dt in ("f32", "bf16"):
        x, u = rows(2, V, dt, 91)
        for s in (dict(), dict(p=0.9), dict(k=30), dict(T=0.0), dict(T=2.0, m=0.01)):
            check(d2, x, u, **s)
    x, u = rows(1, V, "bf16", 93)
    x = x.repeat(256, 1)               # a row per workgroup
    ids, _ = d2.sample(x.to(DEV), torch.tensor(u * 256, device=DEV), top_p=0.99)
    want, _, clear = reference_row(x[0].double().numpy(), 1.0, 0, f32(0.99), 0.0, f32(u[0]))
    assert clear and ids.tolist() == [want] * 256


def test_most_rows_and_longest_row(d2):
    log("sample, most rows")
    R = 1 << 21
    g = torch.Generator(device=DEV).manual_seed(13)
    x = torch.randn(R, 3, generator=g, device=DEV)
    u = torch.rand(R, generator=g, device=DEV)
    top, order = torch.sort(x, dim=1, descending=True, stable=True)
    w = torch.exp(top.double() - top[:, :1].double())
    s = w.cumsum(1)
    gap = (s - (u.double() * s[:, 2])[:, None]).abs().amin(1)
    want = order.gather(1, (s <= (u.double() * s[:, 2])[:, None]).sum(1, keepdim=True))[:, 0]
    ids, _ = d2.sample(x, u)
    sure = gap > 2.0 ** -37
    assert int((~sure).sum()) < 100 and torch.equal(ids[sure].long(), want[sure])
    b = x.bfloat16()
    ids, _ = d2.sample(b, u, temperature=0.0)
    assert torch.equal(ids.long(), torch.sort(b, dim=1, descending=True, stable=True)[1][:, 0])
    del x, b, s, w, top, order
    V = 1 << 24
    for dt in ("f32", "bf16"):
        log(f"sample, longest row {dt}")
        x, u = rows(1, V, dt, 17)
        for kw in (dict(), dict(k=1000, p=0.9)):
            check(d2, x, u, **kw)


def test_extreme_settings(d2):
    x, u = rows(6, 3001, "f32", 8)
    check(d2, x, u, T=[1e-45, 1e-30, 1e30, 3e38, 100.0, 0.001])
    check(d2, x, u, k=[-1, -2 ** 31, 2 ** 31 - 1, 3001, 3000, 3002])
    check(d2, x, u, p=[-1.0, 1.0, 2.0, 1e-30, 1.0 - 2.0 ** -24, 0.5])
    check(d2, x, u, m=[-1.0, 0.0, 5.0, 1e-30, 1.0, 0.999])
    # not numbers: greedy; no cut; u = 0
    nan = math.nan
    ids, _ = d2.sample(x.to(DEV), torch.full((6,), nan, device=DEV))
    top = x.argmax(dim=1).tolist()
    assert ids.tolist() == top
    ids, _ = d2.sample(x.to(DEV), torch.tensor(u, device=DEV), torch.full((6,), nan, device=DEV))
    assert ids.tolist() == top
    want, _ = d2.sample(x.to(DEV), torch.tensor(u, device=DEV))
    got, _ = d2.sample(x.to(DEV), torch.tensor(u, device=DEV), top_p=torch.full((6,), nan, device=DEV),
                       min_p=torch.full((6,), nan, device=DEV))
    assert torch.equal(got, want)
    # numbers outside [0, 1)
    lo, _ = d2.sample(x.to(DEV), torch.full((6,), -3.0, device=DEV))
    hi, _ = d2.sample(x.to(DEV), torch.full((6,), 1.0, device=DEV))
    last, _ = d2.sample(x.to(DEV), torch.full((6,), 1.0 - 2.0 ** -24, device=DEV))
    assert lo.tolist() == top and torch.equal(hi, last)


def test_draws_follow_the_distribution(d2):
    """Stratified uniforms reproduce each token's share to within one stratum."""
    V, n = 13, 4096
    g = torch.Generator().manual_seed(2)
    row = torch.randn(V, generator=g) * 2
    x = row.repeat(n, 1).to(DEV)
    u = (torch.arange(n) + 0.5) / n
    ids, lp = d2.sample(x, u.to(DEV), temperature=1.7)
    want = torch.softmax(row.double() / f32(1.7), 0)
    got = torch.bincount(ids.cpu().long(), minlength=V).double() / n
    assert float((got - want).abs().max()) <= 1.0 / n
    assert torch.allclose(lp.cpu().double().exp(), want[ids.cpu().long()], rtol=1e-6, atol=0)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_random_calls(d2, dt):
    rng = np.random.default_rng(1234 if dt == "f32" else 4321)
    for case in range(24):
        V = int(np.exp(rng.uniform(0, np.log(60000))))
        R = int(rng.integers(1, 6))
        x, u = rows(R, V, dt, int(rng.integers(1 << 30)), spread=float(rng.uniform(0.05, 6)))
        log(f"case {case}: R={R} V={V} {dt}")
        check(d2, x, u, T=rng.choice([0.0, 0.3, 0.8, 1.0, 2.5], R),
              k=rng.choice([0, 1, 7, 64, 1000, 5000], R), p=rng.choice([1.0, 0.3, 0.9, 0.999], R),
              m=rng.choice([0.0, 0.01, 0.3], R))


def test_outputs_and_neighbours(d2):
    """Outputs land where they belong and nowhere else; the same inputs give the same bits."""
    x, u = rows(37, 4099, "bf16", 5)
    ids = torch.full((64,), -7, dtype=torch.int32, device=DEV)
    lp = torch.full((64,), 7.0, device=DEV)
    first = None
    for _ in range(3):
        check(d2, x, u, T=0.9, p=0.97, out=(ids[8:45], lp[8:45]))
        assert bool((ids[:8] == -7).all()) and bool((ids[45:] == -7).all())
        assert bool((lp[:8] == 7).all()) and bool((lp[45:] == 7).all())
        got = (ids.clone(), lp.clone())
        if first is not None:
            assert torch.equal(first[0], got[0]) and torch.equal(first[1], got[1])
        first = got


def test_graph_replay(d2):
    R, V = 20, 90011
    a, ua = rows(R, V, "bf16", 51)
    b, ub = rows(R, V, "bf16", 52)
    dev = lambda x, u: (x.to(DEV), torch.tensor(u, device=DEV))
    a, b = dev(a, ua), dev(b, ub)
    k = torch.tensor([0, 5, 50, 1000] * 5, dtype=torch.int32, device=DEV)
    buf = [t.clone() for t in a]
    d2.sample(*buf, temperature=0.9, top_k=k)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ids, lp = d2.sample(*buf, temperature=0.9, top_k=k)
    for src in (a, b, a, b):
        for t, x in zip(buf, src):
            t.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        want = d2.sample(*src, temperature=0.9, top_k=k)
        torch.cuda.synchronize()
        assert torch.equal(ids, want[0]) and torch.equal(lp, want[1])


def test_two_streams(d2):
    a, ua = rows(30, 95011, "bf16", 61)
    b, ub = rows(9, 50000, "f32", 62)
    a, b = (a.to(DEV), torch.tensor(ua, device=DEV)), (b.to(DEV), torch.tensor(ub, device=DEV))
    wa, wb = d2.sample(*a, top_p=0.95), d2.sample(*b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s1):
            ga = d2.sample(*a, top_p=0.95)
        with torch.cuda.stream(s2):
            gb = d2.sample(*b)
        torch.cuda.synchronize()
        for g, w in ((ga, wa), (gb, wb)):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


def test_binding_rejects(d2):
    x, u = torch.zeros(4, 10, device=DEV), torch.zeros(4, device=DEV)
    for kw in (dict(temperature=torch.ones(3, device=DEV)),
               dict(temperature=torch.ones(4, device=DEV, dtype=torch.float64)),
               dict(top_k=torch.ones(4, device=DEV)), dict(top_p=torch.ones(4)),
               dict(out=(torch.zeros(4, device=DEV), torch.zeros(4, device=DEV)))):
        with pytest.raises(ValueError):
            d2.sample(x, u, **kw)
    with pytest.raises(ValueError):
        d2.sample(x, u[:3])
    with pytest.raises(ValueError):
        d2.sample(x[:, ::2], u)
    with pytest.raises(ValueError):
        d2.sample(x[0], u[:1])
    with pytest.raises(TypeError):
        d2.sample(x.half(), u)
    with pytest.raises(d2.Dflash2Error):
        d2.sample(x, u, temperature=-1.0)
    with pytest.raises(d2.Dflash2Error):
        d2.sample(x[:0], u[:0])
