"""Sampling with a min_p near the least weight that counts, 2^-64 (needs an MI355X).

V = 2^26: the general path's factors have 36 bits behind the point, so a kept mass errs by less than
EPS = 2^-36 of itself, and logprob (a quotient's logarithm, near 0 here) by less than 2 EPS.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
V, EPS = 1 << 26, 2.0 ** -36


def test_a_small_min_p_cuts():
    """Many tokens below a small min_p: their mass, 2^-34.5, is more than the row's precision, and none
    of it is kept. Below them it cuts nothing."""
    import dflash2_draft_candidate_amd as d2
    x = torch.full((1, V), -60.5 * math.log(2), device=DEV)
    x[0, 12345] = 0.0
    u = torch.tensor([0.5], device=DEV)
    for min_p, rest in ((2.0 ** -60.25, 0.0), (2.0 ** -60.75, (V - 1) * 2.0 ** -60.5)):
        ids, lp = d2.sample(x, u, min_p=min_p)
        assert int(ids) == 12345 and abs(float(lp) + rest) <= 2 * EPS
