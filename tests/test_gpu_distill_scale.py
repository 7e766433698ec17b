"""Gradients whose scale g tau passes the largest fp32 number while the gradient itself does not (needs
an MI355X). Tolerances, reference and `check` are those of test_gpu_distill.

With K equal teacher entries p = 1 / K and q < 1 / K, so |g tau (q - p)| < g tau / K.
"""
import math
import sys

import pytest
import torch

from test_gpu_distill import DEV, WAYS, check, inputs, reference, run_all
from test_gpu_sample import f32

pytestmark = pytest.mark.gpu


def log(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("R,V", WAYS + [(140, 170001)])
def test_large_scale(R, V, dt):
    import dflash2_draft_candidate_amd as d2
    log(f"distill, large scale R={R} V={V} {dt}")
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    K = 64
    for tau, size in ((1e20, 1e20), (2.0, 3e38), (1e38, 100.0), (1e-20, 1e-10)):
        tau = f32(tau)  # (the temperature is passed in fp32)
        z, ids, t, g = inputs(R, V, K, dtype, 43)
        t.zero_()
        g = torch.where(g > 0, 1.0, -1.0) * size
        z[2, V // 2:] = -math.inf      # masked tokens: gradient 0
        ids[2] = torch.arange(K, device=DEV)
        z[3] = torch.finfo(dtype).min  # a row of masks
        ids[4] = -1
        ref = reference(z, ids, t, g, tau)
        for loss, grad in run_all(d2, z, ids, t, g, tau):
            assert bool(torch.isfinite(grad).all())
            assert bool((grad[2, V // 2:] == 0).all()) and bool((grad[4] == 0).all())
            check(None, grad, ref, V, tau, g, dtype)


@pytest.mark.parametrize("R,V", WAYS)
def test_infinite_teacher_logit(R, V):
    """+inf among the teacher's logits: the row's loss is NaN, and so is its gradient at the entries;
    everywhere else, and in the other rows, the results are what they are without it."""
    import dflash2_draft_candidate_amd as d2
    K, tau = 5, 1.5
    z, ids, t, g = inputs(R, V, K, torch.float32, 44)
    ref = reference(z, ids, t, g, tau)
    plain = run_all(d2, z, ids, t, g, tau)
    t[3, 2] = math.inf
    t[5] = math.inf
    good = [r for r in range(R) if r not in (3, 5)]
    for (loss, grad), (_, whole) in zip(run_all(d2, z, ids, t, g, tau), plain):
        assert bool(torch.isnan(loss[[3, 5]]).all())
        for r in (3, 5):
            nan = torch.zeros(V, dtype=torch.bool, device=DEV)
            nan[ids[r].long()] = True
            assert torch.equal(torch.isnan(grad[r]), nan)
            assert torch.equal(grad[r][~nan], whole[r][~nan])
        check(loss[good], grad[good], tuple(x[good] for x in ref), V, tau, g[good], torch.float32)
