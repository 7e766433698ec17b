"""The global gradient norm and clipping vs 64 bits (needs an MI355X).

The norm is a 64-bit sum, a square root and one rounding to fp32: u = 2^-24 of itself, and 2 n 2^-53
for the sum of n squares (below u / 16 for n < 2^24). A clipped element is one product in fp32 by a
factor rounded to fp32 (2 u) and the rounding to its type (2^-8 in bf16, u in f32); subnormal results
are off by half of the smallest step (1e-38 covers both types' where they are flushed).
"""
import math
import random
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


def log(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module")
def d2():
    import dflash2_draft_candidate_amd
    return dflash2_draft_candidate_amd


def norm64(grads):
    return math.sqrt(math.fsum(float((g.double() ** 2).sum()) for g in grads))


def make(shapes, seed, scale=1.0):
    """Gradients that are views starting `before` elements into their storage, among guards."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    grads, wholes = [], []
    for shape, dtype, before in shapes:
        n = math.prod(shape)
        whole = (torch.randn(before + n + 9, generator=gen, device=DEV) * scale).to(dtype)
        wholes.append(whole)
        grads.append(whole[before:before + n].view(shape))
    return grads, wholes


def check(d2, shapes, seed=1, scale=1.0, part=0.3):
    grads, wholes = make(shapes, seed, scale)
    before = [w.clone() for w in wholes]
    want = norm64(grads)
    norm = d2.grad_norm(grads)
    assert norm.shape == () and norm.dtype == F32
    assert abs(float(norm) - want) <= 2 * U * want
    limit = torch.tensor(part * want, dtype=F32).item()
    outs, out_wholes = make(shapes, seed + 1)
    out_before = [w.clone() for w in out_wholes]
    got = d2.clip_grads(grads, limit, out=outs)
    assert torch.equal(got, norm)
    assert all(torch.equal(a, b) for a, b in zip(wholes, before))  # inputs, guards: as they were
    f = min(1.0, limit / want) if want > 0 else 1.0
    for g, o, w, b, (shape, dtype, at) in zip(grads, outs, out_wholes, out_before, shapes):
        half = U if dtype == F32 else 2.0 ** -8
        y = g.double() * f
        assert bool(((o.double() - y).abs() <= (half + 3 * U) * y.abs() + 1e-38).all())
        n = math.prod(shape)
        assert torch.equal(w[:at], b[:at]) and torch.equal(w[at + n:], b[at + n:])
    got = d2.clip_grads(grads, limit)
    assert torch.equal(got, norm)
    assert all(torch.equal(g, o) for g, o in zip(grads, outs))
    for w, b, (shape, _, at) in zip(wholes, before, shapes):
        n = math.prod(shape)
        assert torch.equal(w[:at], b[:at]) and torch.equal(w[at + n:], b[at + n:])


@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 255, 2047, 2048, 2049, 8191, 32768, 32769, 100003,
                               5000011])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_sizes(d2, n, dtype):
    log(f"grad norm n={n} {dtype}")
    for before in (0, 1, 3):
        check(d2, [((n,), dtype, before)], seed=n + before)


@pytest.mark.parametrize("count", [1, 2, 127, 128, 129, 300, 1025])
def test_many_tensors(d2, count):
    log(f"grad norm count={count}")
    rng = random.Random(count)
    shapes = [((rng.choice([0, 1, 5, 64, 777, 4096, 30000]),), rng.choice([BF16, F32]),
               rng.randrange(8)) for _ in range(count - 1)] + [((33, 129), BF16, 1)]
    check(d2, shapes, seed=count)


def test_most_tensors(d2):
    """Every launch's partial sums have a place: the most tensors that a call takes."""
    log("grad norm, most tensors")
    count = 1 << 16
    base = torch.randn(2 * count, device=DEV)
    grads = [base[2 * i:2 * i + 1 + i % 2] for i in range(count)]
    want = norm64([torch.cat(grads)])
    norm = d2.grad_norm(grads)
    assert abs(float(norm) - want) <= 2 * U * want
    copy = base.clone()
    d2.clip_grads(grads, want / 2)
    used = torch.ones(2 * count, dtype=torch.bool, device=DEV)
    used[1::4] = False
    assert torch.equal(base[~used], copy[~used])
    y = copy[used].double() / 2
    assert bool(((base[used].double() - y).abs() <= 6 * U * y.abs() + 1e-38).all())


@pytest.mark.parametrize("scale", [1e-30, 1e-22, 1e18, 3e37])
def test_range(d2, scale):
    """Squares far outside fp32."""
    n = 100 if scale > 1e30 else 5000  # (the norm itself stays a float)
    check(d2, [((n,), F32, 0), ((n,), BF16, 1)], scale=scale / 6)


def test_nothing_to_clip(d2):
    for part in (1.0001, 5.0):
        check(d2, [((3000,), F32, 0), ((70000,), BF16, 1)], part=part)
    zeros = [torch.zeros(5000, device=DEV), torch.zeros(77, dtype=BF16, device=DEV)]
    for limit in (0.0, 1.0):
        assert float(d2.clip_grads(zeros, limit)) == 0.0
        assert all(bool((z == 0).all()) for z in zeros)
    empty = [torch.empty(0, device=DEV), torch.empty(0, 5, dtype=BF16, device=DEV)]
    assert float(d2.grad_norm(empty)) == 0.0 and float(d2.clip_grads(empty, 1.0)) == 0.0
    g = torch.randn(5000, device=DEV)
    d2.clip_grads(g, 0.0)
    assert bool((g == 0).all())


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_not_finite(d2, bad):
    """A norm that is not finite scales nothing."""
    grads, _ = make([((3000,), F32, 0), ((70000,), BF16, 1)], 3)
    grads[1][69999] = bad
    before = [g.clone() for g in grads]
    outs = [torch.zeros_like(g) for g in grads]
    for out in (None, outs):
        norm = d2.clip_grads(grads, 0.5, out=out)
        assert math.isnan(float(norm)) if math.isnan(bad) else float(norm) == math.inf
        for g, b in zip(grads if out is None else outs, before):
            assert torch.equal(g.isnan(), b.isnan())
            assert torch.equal(g.nan_to_num(0.0), b.nan_to_num(0.0))
    big = [torch.full((300,), 3e38, device=DEV)]  # past the largest float
    assert float(d2.clip_grads(big, 1.0)) == math.inf and float(big[0][0]) == torch.tensor(3e38)


def test_graph_replay(d2):
    grads, _ = make([((3000,), F32, 1), ((70000,), BF16, 3), ((4096, 64), BF16, 0)], 7)
    outs = [torch.empty_like(g) for g in grads]
    d2.clip_grads(grads, 1.0, out=outs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = d2.clip_grads(grads, 1.0, out=outs)
    for i in range(4):
        for g in grads:
            g.copy_(torch.randn(g.shape, device=DEV) * (0.001 + 0.1 * i))
        graph.replay()
        torch.cuda.synchronize()
        want = [torch.empty_like(g) for g in grads]
        assert torch.equal(d2.clip_grads(grads, 1.0, out=want), norm)
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_streams(d2):
    a = make([((500000,), BF16, 1)], 9)[0]
    b = make([((3000,), F32, 0)] * 200, 10)[0]
    na, nb = d2.grad_norm(a), d2.grad_norm(b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s1):
            ga = d2.grad_norm(a)
        with torch.cuda.stream(s2):
            gb = d2.grad_norm(b)
        torch.cuda.synchronize()
        assert torch.equal(ga, na) and torch.equal(gb, nb)


def test_outputs_side_by_side(d2):
    """Outputs that touch, in any order, and gradients named twice: fine; twice the same output: refused,
    and nothing is written."""
    gen = torch.Generator(device=DEV).manual_seed(9)
    flat = torch.zeros(1000, device=DEV)
    g = [torch.randn(n, generator=gen, device=DEV) for n in (300, 1, 0, 699)]
    out = [flat[700:], flat[699:700], flat[:0], flat[:699]]
    norm = d2.clip_grads(g, 1.0, out=out)
    want = math.sqrt(sum(float((x.double() ** 2).sum()) for x in g))
    assert abs(float(norm) - want) <= 2.0 ** -23 * want
    for x, y in zip(g, out):
        assert bool(((y.double() - x.double() / want).abs() <= 2.0 ** -22 * x.double().abs() / want).all())
    twice = d2.clip_grads([g[0], g[0]], 1.0, out=[flat[:300], flat[300:600]])
    want = math.sqrt(2.0 * float((g[0].double() ** 2).sum()))
    assert abs(float(twice) - want) <= 2.0 ** -23 * want and torch.equal(flat[:300], flat[300:600])
    before = g[0].clone()
    for grads, o in (([g[0], g[0]], None), ([g[0], g[0][10:20]], None), ([g[0], g[3]], [g[3][:300], flat[:699]])):
        with pytest.raises(d2.Dflash2Error):
            d2.clip_grads(grads, 1e-3, out=o)
    assert torch.equal(before, g[0])
