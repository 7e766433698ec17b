"""Clipping by factors that are no normal float (needs an MI355X).

max_norm / norm may lie far below 2^-126 while gradients and results are ordinary floats: the result is
the product rounded to the type, as for any factor. With u = 2^-24: the quotient and the product in 64
bits err by 2^-50 at most, the norm that the quotient is taken by as much; then a rounding to fp32 (u) and
one to bf16 (2^-8), and half of the smallest step where results are subnormal (1e-38 where flushed).
"""
import math
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def d2():
    import dflash2_draft_candidate_amd
    return dflash2_draft_candidate_amd


@pytest.mark.parametrize("n", [1, 77, 5003, 300001])
@pytest.mark.parametrize("scale,max_norm", [
    (3e37, 1e-3), (1e36, 1e-2), (1e35, 1e-6), (1e35, 1e-9), (1e35, 1e-30), (1e30, 1e-12), (1e20, 1e-18),
    (1e20, 1e-19), (1.0, 3e-38), (1e-3, 1e-40), (1e35, 0.0)])
def test_small_factors(d2, n, scale, max_norm):
    print(f"clip factor n={n} scale={scale} max_norm={max_norm}", file=sys.stderr, flush=True)
    gen = torch.Generator(device=DEV).manual_seed(n)
    scale = scale / math.sqrt(n)
    # (views that start anywhere; values over some binades)
    wholes = [(torch.randn(n + 3, generator=gen, device=DEV) * scale * 2.0 ** (i % 3)).to(t)
              for i, t in enumerate((F32, BF16, BF16, F32))]
    grads = [w[1:n + 1] for w in wholes]
    limit = torch.tensor(max_norm, dtype=F32).item()  # (it is passed in fp32)
    want = math.sqrt(math.fsum(float((g.double() ** 2).sum()) for g in grads))
    outs = [torch.full_like(w, 7.0) for w in wholes]
    norm = d2.clip_grads(grads, limit, out=[o[1:n + 1] for o in outs])
    assert abs(float(norm) - want) <= 2 * U * want < math.inf
    f = min(1.0, limit / want)
    for g, w, o in zip(grads, wholes, outs):
        half = (U if g.dtype == F32 else 2.0 ** -8) + 2 * U
        y = g.double() * f
        assert bool(((o[1:n + 1].double() - y).abs() <= half * y.abs() + 1e-38).all())
        assert float(o[0]) == 7.0 and bool((o[n + 1:] == 7).all())
    d2.clip_grads(grads, limit)  # in place: the same
    assert all(torch.equal(g, o[1:n + 1]) for g, o in zip(grads, outs))
