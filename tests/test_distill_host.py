"""Refusals of the distillation entry points, on the host: every call fails validation before
anything is launched (the pointers are fake)."""
import ctypes

import pytest
import torch

OK, EINVAL, EUNSUP, EALIGN, EWS, EHIP = 0, -1, -2, -3, -4, -5
F32, BF16 = 0, 1
P = 0x100000     # fake, 16-byte aligned, never dereferenced
Q = 0x900000000  # another one, far from P
MIS = 0x100008


@pytest.fixture(scope="module")
def d2():
    import dflash2_draft_candidate_amd
    return dflash2_draft_candidate_amd


SIZES = [
    (dict(dt=2), EINVAL), (dict(dt=-1), EINVAL), (dict(R=0), EINVAL), (dict(R=-1), EINVAL),
    (dict(R=(1 << 21) + 1), EINVAL), (dict(V=0), EINVAL), (dict(V=(1 << 28) + 1), EINVAL),
    (dict(K=0), EINVAL), (dict(K=65), EINVAL), (dict(tau=0.0), EINVAL), (dict(tau=-1.0), EINVAL),
    (dict(tau=float("nan")), EINVAL), (dict(tau=float("inf")), EINVAL), (dict(tau=1e-40), EINVAL),
    (dict(student=None), EINVAL), (dict(ids=None), EINVAL), (dict(t=None), EINVAL),
    (dict(student=MIS), EALIGN), (dict(ids=MIS), EALIGN), (dict(t=MIS), EALIGN),
]


def args(kw):
    a = dict(student=P, dt=BF16, ids=P, t=P, R=16, V=151936, K=8, tau=1.0, loss=Q, stats=Q, g=P,
             grad=Q, ws=P, wsb=0)
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(loss=None), EINVAL), (dict(stats=None), EINVAL), (dict(loss=MIS), EALIGN),
    (dict(stats=MIS), EALIGN), (dict(), EWS), (dict(ws=None, wsb=1 << 30), EWS),
    (dict(ws=MIS, wsb=1 << 30), EALIGN)])
def test_forward_rejects(d2, kw, status):
    a = args(kw)
    assert d2.library().dflash2_distill(a["student"], a["dt"], a["ids"], a["t"], a["R"], a["V"],
                                        a["K"], a["tau"], a["loss"], a["stats"], a["ws"],
                                        a["wsb"], None) == status


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(g=None), EINVAL), (dict(grad=None), EINVAL), (dict(g=MIS), EALIGN),
    (dict(grad=MIS), EALIGN), (dict(stats=None), EINVAL), (dict(stats=MIS), EALIGN),
    (dict(grad=P), EINVAL), (dict(grad=P + 16 * 151936 * 2 - 16), EINVAL)])
def test_backward_rejects(d2, kw, status):
    a = args(kw)
    assert d2.library().dflash2_distill_backward(a["student"], a["dt"], a["ids"], a["t"],
                                                 a["stats"], a["g"], a["R"], a["V"], a["K"],
                                                 a["tau"], a["grad"], None) == status


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(g=None), EINVAL), (dict(grad=None), EINVAL), (dict(loss=None), EINVAL),
    (dict(g=MIS), EALIGN), (dict(grad=MIS), EALIGN), (dict(loss=MIS), EALIGN), (dict(), EWS),
    (dict(grad=P), EINVAL), (dict(grad=P + 4096), EINVAL), (dict(ws=MIS, wsb=1 << 30), EALIGN)])
def test_step_rejects(d2, kw, status):
    a = args(kw)
    assert d2.library().dflash2_distill_step(a["student"], a["dt"], a["ids"], a["t"], a["g"],
                                             a["R"], a["V"], a["K"], a["tau"], a["loss"],
                                             a["grad"], a["ws"], a["wsb"], None) == status


def test_workspace_sizes(d2):
    f = d2.library().dflash2_distill_workspace_bytes
    assert f(16, 151936, BF16) > 0      # few rows: slices
    assert f(0, 151936, BF16) == 0
    assert f(16, 151936, 7) == 0
    assert f((1 << 21) + 1, 8, F32) == 0


def test_binding_rejects(d2):
    z, i, t = torch.zeros(2, 10), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3)
    g = torch.zeros(2)
    for call in (lambda: d2.distill(z, i, t),
                 lambda: d2.distill_backward(z, i, t, torch.zeros(2, 2), g),
                 lambda: d2.distill_step(z, i, t, g),
                 lambda: d2.distill_loss(z, i, t)):
        with pytest.raises(ValueError):  # tensors on the host
            call()
    with pytest.raises(ValueError):
        d2.distill_loss(z, i, t.requires_grad_())
