"""Refusals of the gradient norm and of clipping, on the host: every call fails validation before
anything is launched (the device pointers are fake)."""
import ctypes

import pytest
import torch

OK, EINVAL, EUNSUP, EALIGN, EWS, EHIP = 0, -1, -2, -3, -4, -5
F32, BF16 = 0, 1
P, Q = 0x100000, 0x900000000
WS = 1 << 20


@pytest.fixture(scope="module")
def d2():
    import dflash2_draft_candidate_amd
    return dflash2_draft_candidate_amd


CASES = [
    (dict(count=-1), EINVAL), (dict(count=(1 << 16) + 1), EINVAL), (dict(grads=None), EINVAL),
    (dict(sizes=None), EINVAL), (dict(dtypes=None), EINVAL), (dict(dtypes=[F32, 2]), EINVAL),
    (dict(sizes=[8, -1]), EINVAL), (dict(sizes=[8, (1 << 40) + 1]), EINVAL),
    (dict(sizes=[1 << 40, 1]), EINVAL), (dict(grads=[P, 0]), EINVAL), (dict(grads=[P + 2, P]), EALIGN),
    (dict(grads=[P, P + 1]), EALIGN), (dict(norm=None), EINVAL), (dict(norm=P + 4), EALIGN),
    (dict(wsb=0), EWS), (dict(ws=None), EWS), (dict(ws=P + 8), EALIGN),
]


def arrays(kw):
    a = dict(grads=[P, P + 4096], sizes=[8, 8], dtypes=[F32, BF16], out=[P, Q], count=2, norm=Q,
             ws=P, wsb=WS, max_norm=1.0)
    a.update(kw)
    keep = []
    for name, kind in (("grads", ctypes.c_uint64), ("sizes", ctypes.c_int64),
                       ("dtypes", ctypes.c_int32), ("out", ctypes.c_uint64)):
        if a[name] is not None:
            arr = (kind * len(a[name]))(*a[name])
            keep.append(arr)
            a[name] = ctypes.addressof(arr)
    return a, keep


@pytest.mark.parametrize("kw,status", CASES)
def test_norm_rejects(d2, kw, status):
    a, keep = arrays(kw)
    assert d2.library().dflash2_grad_norm(a["grads"], a["sizes"], a["dtypes"], a["count"],
                                          a["norm"], a["ws"], a["wsb"], None) == status


@pytest.mark.parametrize("kw,status", CASES + [
    (dict(out=None), EINVAL), (dict(out=[P, 0]), EINVAL), (dict(out=[P + 16, Q]), EINVAL),
    (dict(out=[P, P + 4096 - 2]), EINVAL), (dict(out=[P, Q + 1]), EALIGN),
    (dict(out=[Q + 2, Q]), EALIGN), (dict(max_norm=-1.0), EINVAL),
    # an output that overlaps another one, or a gradient that is not its own
    (dict(out=[Q, Q]), EINVAL), (dict(out=[Q, Q + 30]), EINVAL), (dict(out=[Q + 12, Q]), EINVAL),
    (dict(out=[P + 4096, Q]), EINVAL), (dict(out=[P + 4096 - 28, Q]), EINVAL),
    (dict(out=[Q, P + 30]), EINVAL), (dict(out=[P, P]), EINVAL),
    (dict(grads=[P, P], dtypes=[F32, F32], out=[P, P]), EINVAL),
    (dict(grads=[P, P], dtypes=[F32, F32], out=[Q, P]), EINVAL),
    (dict(grads=[P, P + 16], dtypes=[F32, F32], out=[P, P + 16]), EINVAL),
    (dict(max_norm=float("nan")), EINVAL), (dict(max_norm=float("inf")), EINVAL)])
def test_clip_rejects(d2, kw, status):
    a, keep = arrays(kw)
    assert d2.library().dflash2_clip_grads(a["grads"], a["sizes"], a["dtypes"], a["count"],
                                           a["out"], a["max_norm"], a["norm"], a["ws"], a["wsb"],
                                           None) == status


def test_binding_rejects(d2):
    g = [torch.zeros(4), torch.zeros(3, dtype=torch.bfloat16)]
    for call in (lambda: d2.grad_norm(g), lambda: d2.clip_grads(g, 1.0), lambda: d2.grad_norm([]),
                 lambda: d2.clip_grads([], 1.0)):
        with pytest.raises(ValueError):  # tensors on the host, none at all
            call()
