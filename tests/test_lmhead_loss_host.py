"""Refusals of the LM head's losses, on the host: every call fails validation before anything is
launched (the pointers are fake)."""
import pytest
import torch

OK, EINVAL, EUNSUP, EALIGN, EWS, EHIP = 0, -1, -2, -3, -4, -5
F32, BF16 = 0, 1
P = 0x100000        # fake, 16-byte aligned, never dereferenced
A, B = 0x90000000000, 0xA0000000000  # others, far from P and from each other
MIS = 0x100008


@pytest.fixture(scope="module")
def d2():
    import dflash2_draft_candidate_amd
    return dflash2_draft_candidate_amd


SIZES = [
    (dict(dt=2), EINVAL), (dict(dt=-1), EINVAL), (dict(R=0), EINVAL), (dict(R=-1), EINVAL),
    (dict(R=(1 << 16) + 1), EINVAL), (dict(V=0), EINVAL), (dict(V=(1 << 28) + 1), EINVAL),
    (dict(H=0), EINVAL), (dict(H=4), EINVAL), (dict(H=12), EINVAL), (dict(H=(1 << 16) + 8), EINVAL),
    (dict(hidden=None), EINVAL), (dict(W=None), EINVAL), (dict(ids=None), EINVAL),
    (dict(hidden=MIS), EALIGN), (dict(W=MIS), EALIGN), (dict(ids=MIS), EALIGN),
    (dict(stats=None), EINVAL), (dict(stats=MIS), EALIGN),
]
DISTILL = [
    (dict(K=0), EINVAL), (dict(K=65), EINVAL), (dict(tau=0.0), EINVAL), (dict(tau=-1.0), EINVAL),
    (dict(tau=float("nan")), EINVAL), (dict(tau=float("inf")), EINVAL), (dict(tau=1e-40), EINVAL),
    (dict(t=None), EINVAL), (dict(t=MIS), EALIGN),
]
FORWARD = [
    (dict(loss=None), EINVAL), (dict(loss=MIS), EALIGN), (dict(), EWS),
    (dict(ws=None, wsb=1 << 40), EWS), (dict(ws=MIS, wsb=1 << 40), EALIGN),
]
BACKWARD = [
    (dict(g=None), EINVAL), (dict(g=MIS), EALIGN), (dict(gh=None, gw=None), EINVAL),
    (dict(gh=MIS), EALIGN), (dict(gw=MIS), EALIGN), (dict(gh=P), EINVAL), (dict(gw=P), EINVAL),
    (dict(gw=P + 64 * 1000 * 2 - 16), EINVAL), (dict(gh=B + 4096), EINVAL), (dict(), EWS),
    (dict(gh=None), EWS), (dict(gw=None), EWS), (dict(ws=None, wsb=1 << 40), EWS),
    (dict(ws=MIS, wsb=1 << 40), EALIGN),
]


def args(kw):
    a = dict(hidden=P, W=P, dt=BF16, ids=P, t=P, R=16, H=64, V=1000, K=8, tau=1.0, loss=A, stats=P,
             g=P, gh=A, gw=B, ws=P, wsb=0)
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,status", SIZES + FORWARD)
def test_ce_rejects(d2, kw, status):
    a = args(kw)
    assert d2.library().dflash2_lmhead_ce(
        a["hidden"], a["W"], a["dt"], a["ids"], a["R"], a["H"], a["V"], a["loss"], a["stats"],
        a["ws"], a["wsb"], None) == status


@pytest.mark.parametrize("kw,status", SIZES + DISTILL + FORWARD)
def test_distill_rejects(d2, kw, status):
    a = args(kw)
    assert d2.library().dflash2_lmhead_distill(
        a["hidden"], a["W"], a["dt"], a["ids"], a["t"], a["R"], a["H"], a["V"], a["K"], a["tau"],
        a["loss"], a["stats"], a["ws"], a["wsb"], None) == status


@pytest.mark.parametrize("kw,status", SIZES + BACKWARD)
def test_ce_backward_rejects(d2, kw, status):
    a = args(kw)
    assert d2.library().dflash2_lmhead_ce_backward(
        a["hidden"], a["W"], a["dt"], a["ids"], a["stats"], a["g"], a["R"], a["H"], a["V"],
        a["gh"], a["gw"], a["ws"], a["wsb"], None) == status


@pytest.mark.parametrize("kw,status", SIZES + DISTILL + BACKWARD)
def test_distill_backward_rejects(d2, kw, status):
    a = args(kw)
    assert d2.library().dflash2_lmhead_distill_backward(
        a["hidden"], a["W"], a["dt"], a["ids"], a["t"], a["stats"], a["g"], a["R"], a["H"], a["V"],
        a["K"], a["tau"], a["gh"], a["gw"], a["ws"], a["wsb"], None) == status


def test_workspace_sizes(d2):
    f = d2.library().dflash2_lmhead_loss_workspace_bytes
    for backward in (0, 1):
        assert f(16, 4096, 151936, BF16, backward) > 0
        assert f(0, 4096, 151936, BF16, backward) == 0
        assert f(16, 4095, 151936, BF16, backward) == 0
        assert f(16, 4096, 151936, 7, backward) == 0
    # one piece of G and the rest, whatever the vocabulary: far from the logits
    assert f(4096, 4096, 151936, BF16, 1) < 600 << 20
    assert f(1 << 16, 64, 151936, BF16, 1) < 600 << 20


def test_binding_rejects(d2):
    h, W = torch.zeros(2, 16), torch.zeros(10, 16)
    i, t, g = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3), torch.zeros(2)
    for call in (lambda: d2.lmhead_ce(h, W, i[:, 0]),
                 lambda: d2.lmhead_ce_backward(h, W, i[:, 0], torch.zeros(2, 3), g),
                 lambda: d2.lmhead_ce_loss(h, W, i[:, 0]),
                 lambda: d2.lmhead_distill(h, W, i, t),
                 lambda: d2.lmhead_distill_backward(h, W, i, t, torch.zeros(2, 5), g),
                 lambda: d2.lmhead_distill_loss(h, W, i, t)):
        with pytest.raises(ValueError):  # tensors on the host
            call()
    with pytest.raises(ValueError):
        d2.lmhead_distill_loss(h, W, i, t.requires_grad_())
