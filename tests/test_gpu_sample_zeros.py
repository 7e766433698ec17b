"""Sampling from rows whose largest logits are zeros of both signs and the type's smallest numbers next
to them, more than a list holds (needs an MI355X). The reference, its tolerances and `check` are those
of test_gpu_sample.

All of them weigh 1 to 2^-100, so running sums are whole numbers: the cut's place counts the tokens, zeros
(equal, whatever their sign) before the negative ones. At most of these temperatures the search by value
ends between the two, where the key below zero's is that of -0, which no logit has.
"""
import sys

import pytest
import torch

from test_gpu_sample import check

pytestmark = pytest.mark.gpu

TS = [0.5, 0.7, 0.8, 0.9, 1.0, 1.1, 1.3, 2.0, 3.0, 5.0]


def log(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module")
def d2():
    import dflash2_draft_candidate_amd
    return dflash2_draft_candidate_amd


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("above,zeros,below", [(0, 1500, 600), (0, 1500, 1400), (0, 3, 2500),
                                               (1200, 1500, 1400), (1300, 2, 1300), (700, 0, 5000),
                                               (0, 40, 30)])
def test_zeros_among_the_smallest_numbers(d2, above, zeros, below, dt):
    V, n = 40000, above + zeros + below
    tiny = 2.0 ** -149 if dt == "f32" else 2.0 ** -133
    value = torch.cat([torch.full((above,), tiny), torch.zeros(zeros), torch.full((below,), -tiny)])
    value[above:above + zeros:2] = -0.0
    x = torch.full((6, V), -torch.inf)
    g = torch.Generator().manual_seed(n)
    for r in range(6):
        x[r, torch.randperm(V, generator=g)[:n]] = value
    x = x.to(torch.float32 if dt == "f32" else torch.bfloat16)
    assert bool((x[0][x[0] > -torch.inf] != 0).sum() == above + below)  # nothing was flushed
    # in the first third, at zeros, just behind them, far behind
    u = [0.1, (above + 0.5 * zeros) / n, (above + zeros + 0.5) / n, 0.71, 0.93, 1.0 - 2.0 ** -24]
    u = [min(v, 1.0 - 2.0 ** -24) for v in u]
    for T in TS:
        log(f"zeros {above}/{zeros}/{below} {dt} T={T}")
        check(d2, x, u, T=T)
        check(d2, x, u, T=T, k=above + zeros + below // 2 + 1)
        check(d2, x, u, T=T, p=0.8125)
        check(d2, x, u, T=T, k=n - 1, p=0.96875, m=0.5)
