"""Refusals of dflash2_sample, on the host: every call fails validation before anything is
launched (the pointers are fake)."""
import pytest
import torch

OK, EINVAL, EUNSUP, EALIGN, EWS, EHIP = 0, -1, -2, -3, -4, -5
F32, BF16 = 0, 1
P = 0x100000     # fake, 16-byte aligned, never dereferenced
MIS = 0x100008
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def d2():
    import dflash2_draft_candidate_amd
    return dflash2_draft_candidate_amd


@pytest.mark.parametrize("kw,status", [
    (dict(dt=2), EINVAL), (dict(dt=-1), EINVAL), (dict(R=0), EINVAL), (dict(R=-5), EINVAL),
    (dict(R=(1 << 21) + 1), EINVAL), (dict(V=0), EINVAL), (dict(V=(1 << 28) + 1), EINVAL),
    (dict(t_all=-1.0), EINVAL), (dict(t_all=NAN), EINVAL), (dict(t_all=INF), EINVAL),
    (dict(p_all=NAN), EINVAL), (dict(m_all=NAN), EINVAL), (dict(logits=None), EINVAL),
    (dict(u=None), EINVAL), (dict(ids=None), EINVAL), (dict(logits=MIS), EALIGN),
    (dict(u=MIS), EALIGN), (dict(ids=MIS), EALIGN), (dict(lp=MIS), EALIGN), (dict(t=MIS), EALIGN),
    (dict(k=MIS), EALIGN), (dict(p=MIS), EALIGN), (dict(m=MIS), EALIGN),
    # a value for all rows is not looked at where a tensor takes its place
    (dict(t=MIS, t_all=NAN), EALIGN), (dict(p=MIS, p_all=NAN), EALIGN),
    (dict(m=MIS, m_all=NAN), EALIGN),
    (dict(V=151936), EWS), (dict(V=151936, wsb=16), EWS), (dict(V=151936, ws=None, wsb=1 << 30), EWS),
    (dict(V=151936, ws=MIS, wsb=1 << 30), EALIGN),
])
def test_rejects(d2, kw, status):
    a = dict(logits=P, dt=BF16, R=4, V=100, t=None, t_all=1.0, k=None, k_all=0, p=None, p_all=1.0,
             m=None, m_all=0.0, u=P, ids=P, lp=None, ws=P, wsb=0)
    a.update(kw)
    assert d2.library().dflash2_sample(a["logits"], a["dt"], a["R"], a["V"], a["t"], a["t_all"],
                                       a["k"], a["k_all"], a["p"], a["p_all"], a["m"], a["m_all"],
                                       a["u"], a["ids"], a["lp"], a["ws"], a["wsb"],
                                       None) == status


def test_binding_rejects_host_tensors(d2):
    with pytest.raises(ValueError):
        d2.sample(torch.zeros(2, 10), torch.zeros(2))


def test_workspace_sizes(d2):
    f = d2.library().dflash2_sample_workspace_bytes
    assert f(4, 151936, BF16) > 0        # few rows: slices
    assert f(1024, 151936, BF16) == 0
    assert f(4, 151936, F32) == 0
    assert f(0, 151936, BF16) == 0 and f(4, 0, BF16) == 0 and f(4, 100, 3) == 0
