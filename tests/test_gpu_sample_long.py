"""Sampling from rows of 2^22 logits to the most a row may have (needs an MI355X), against the
definition in 64 bits, computed on the GPU by a sort.

Precision. A general row's bins sum factors with f bits behind the point: 41 up to V = 2^22 - 1, then
one less for each doubling, 62 - floor(log2 V). A weight in such a sum errs by half a step of its factor
(at least 0.989), the factor's polynomial (2^-42.5) and the fp64 roundings of its argument (2^-46): below
2^-40 of itself up to f = 40, below 2^-f from there on (0.506 2^-f + 2^-42.4). So do the sums, and eps is that.
  * A cut compares a running sum with a product of another: either errs by eps of itself, so the answer
    is the reference's unless they are within 2 eps (2.5 here, for the reference's own sums) of the
    row's mass of each other. The inputs have no such place (asserted).
  * logprob: the token's weight and the kept mass, 2 eps, and its rounding to fp32, 2^-24 of itself.
"""
import math
import sys

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


def eps(V):
    return 2.0 ** -min(40, 62 - int(math.floor(math.log2(V))))


def f32(v):
    return float(torch.tensor(v, dtype=torch.float32))


class Row:
    """A row in candidate order, with the running sums of its weights."""

    def __init__(self, x, T):
        self.x, order = torch.sort(x, descending=True, stable=True)
        self.order = order.int()
        del order
        self.w = torch.exp((self.x.double() - self.x[0].double()) / f32(T))
        self.w[self.w < 2.0 ** -64] = 0
        self.N = int((self.w > 0).sum())
        self.S = torch.cumsum(self.w, 0)

    def first(self, target, strictly, n):
        """The first place whose running sum reaches (passes) the target, below n."""
        j = int(torch.searchsorted(self.S, torch.tensor([target], dtype=torch.float64, device=DEV),
                                   right=strictly)[0])
        near = self.S[max(j - 1, 0):j + 1]
        assert float((near - target).abs().min()) > 2.5 * eps(len(self.S)) * float(self.S[-1]), \
            "the inputs leave the answer open"
        return min(j, n - 1)

    def draw(self, u, k=0, p=1.0, m=0.0):
        n = min(k, self.N) if k >= 1 else self.N
        Z = float(self.S[n - 1])
        cuts = [n]
        if p < 1:
            cuts.append(self.first(f32(p) * Z, False, self.N) + 1)
        if m > 0:
            cuts.append(max(1, int((self.w >= min(f32(m), 1.0)).sum())))
        n = min(cuts)
        W = float(self.S[n - 1])
        j = self.first(f32(u) * W, True, n)
        return int(self.order[j]), math.log(float(self.w[j]) / W)


SETTINGS = [dict(), dict(p=0.9), dict(k=1000, p=0.9), dict(k=1500000), dict(m=0.01),
            dict(k=2000000, p=0.5, m=1e-5)]


@pytest.mark.parametrize("V", [(1 << 22) + 3, (1 << 24) - 5, (1 << 26) + 1, 1 << 28])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_long_rows(d2, V, dt):
    log(f"sample, V={V} {dt}")
    g = torch.Generator(device=DEV).manual_seed(V % 1000 + len(dt))
    x = torch.randn(V, generator=g, device=DEV).mul_(3.0)
    x = x if dt == "f32" else x.bfloat16()
    row = Row(x, 0.9)
    u = [0.11, 0.618, 0.9, 0.35, 0.77, 0.5]
    for i, s in enumerate(SETTINGS):
        want, lp = row.draw(u[i], **s)
        ids, got = d2.sample(x[None], torch.tensor(u[i:i + 1], device=DEV), 0.9, s.get("k", 0),
                             s.get("p", 1.0), s.get("m", 0.0))
        log(f"  {s}: {int(ids)}, {float(got)} (expected {want}, {lp})")
        assert int(ids) == want
        assert abs(float(got) - lp) <= 2 * eps(V) + 2.0 ** -24 * abs(lp)
    ids, got = d2.sample(x[None], torch.tensor([0.3], device=DEV), 0.0)
    assert int(ids) == int(row.order[0]) and float(got) == 0.0
