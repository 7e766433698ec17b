"""Sampling with a temperature of +inf in a row's settings, and other very high ones (needs an MI355X):
every logit above -inf weighs the same. Reference and `check` are those of test_gpu_sample; the running
sums are whole numbers, exact on both sides."""
import math
import sys

import pytest
import torch

from test_gpu_sample import check

pytestmark = pytest.mark.gpu

INF = math.inf


def log(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module")
def d2():
    import dflash2_draft_candidate_amd
    return dflash2_draft_candidate_amd


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("V", [700, 20011, 90000])
def test_infinite_temperature(d2, V, dt):
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    g = torch.Generator().manual_seed(V)
    x = torch.randn(6, V, generator=g) * 3
    x[1, ::2] = -INF
    x[2, 5:] = torch.finfo(dtype).min
    x[3] = -INF
    x[3, V // 2] = -3.0
    x[4, ::3] = math.nan
    x[5, V // 3] = 1e30
    x = x.to(dtype)
    T = [INF] * 6
    u = [0.0, 0.31, 0.5, 0.77, 0.93, 1.0 - 2.0 ** -24]
    for s in (dict(), dict(k=300), dict(p=0.40625), dict(k=500, p=0.75), dict(m=1.0), dict(k=V - 1)):
        log(f"T=inf V={V} {dt} {s}")
        check(d2, x, u, T=T, **s)
