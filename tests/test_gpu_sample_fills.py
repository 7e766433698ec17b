"""Sampling from rows that hold one value very often, near the ends of the general path's bins (needs
an MI355X). The reference, its tolerances and `check` are those of test_gpu_sample.

A general row's bins are 32 to an octave of weight and end 88 octaves (60.98 in units of T) below the
first pass's reference, or 127 octaves (88.01) below the maximum after a second pass. A token that
far down has no weight to speak of, however many there are: the answer is the token above.
"""
import math
import sys

import pytest
import torch

from test_gpu_sample import check

pytestmark = pytest.mark.gpu

U = [0.0, 0.37, 0.5, 1.0 - 2.0 ** -24]


def log(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module")
def d2():
    import dflash2_draft_candidate_amd
    return dflash2_draft_candidate_amd


def depths(last_bin):
    """Distances from the reference, in units of T, of places in and around the last bin (its middle is
    `last_bin` / 32 octaves down)."""
    return [(last_bin + o) / 32 * math.log(2) for o in
            (-1.0, -0.51, -0.49, -0.01, 0.01, 0.25, 0.45, 0.49, 0.51, 1.0)]


SETTINGS = [dict(), dict(k="V"), dict(p=1.0, m=0.0), dict(p=0.9), dict(k=3), dict(m=0.01)]


def run(d2, x, T):
    V = x.shape[1]
    for s in SETTINGS:
        s = {a: V if b == "V" else b for a, b in s.items()}
        check(d2, x, (U * len(x))[:len(x)], T=T, **s)


@pytest.mark.parametrize("T,top", [(1.0, 0.0), (0.7, 10.6875)])
@pytest.mark.parametrize("at", [8000, 39000])  # among the first logits read, or above the reference
def test_fill_at_the_ends_of_the_bins(d2, at, T, top):
    # (first pass: headroom 1280 bins above the reference, the last bin's middle 4095 - 1280 below it;
    # a second pass leaves 32 bins above the maximum)
    last = 2815 if at == 8000 else 4063
    R = len(depths(last))
    x = torch.empty(R, 40000)
    for r, d in enumerate(depths(last)):
        x[r] = top - d * T
    x[:, at] = top
    x[:, at + 1:at + 4] = top - 1.5
    log(f"fill below {top} at T={T}, maximum at {at}")
    run(d2, x, T)


@pytest.mark.parametrize("V", [40000, 80000])  # a workgroup per row; slices
@pytest.mark.parametrize("at", [3000, 39000])
def test_fill_in_bf16_rows(d2, at, V):
    """A logit of 300 sends these rows to the general path; T puts the fill where it is wanted."""
    last = 2815 if at == 3000 else 4063
    x = torch.full((4, V), -32.0)
    x[:, at] = 300.0
    x[:, at + 1] = 298.0
    for d in depths(last):
        log(f"bf16 fill {d} T below the maximum, V={V}, maximum at {at}")
        run(d2, x.bfloat16(), 332.0 / d)


def test_fill_as_given(d2):
    """The plain case: one token, the rest filled with a finite number."""
    x = torch.full((4, 40000), -60.98)
    x[:, 8000] = 0.0
    check(d2, x, U)
    x = torch.full((4, 40000), -32.0)
    x[:, 8000] = 10.6875
    check(d2, x, U, T=0.7)
