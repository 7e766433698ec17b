"""Clipping and autograd (needs an MI355X): tensors that are written count as written, so a graph that has
saved one refuses its backward pass, as after any of torch's own in-place operations."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def d2():
    import dflash2_draft_candidate_amd
    return dflash2_draft_candidate_amd


def test_written_tensors_count_as_written(d2):
    w = torch.randn(1000, device=DEV, requires_grad=True)
    grad, = torch.autograd.grad((w ** 3).sum(), w, create_graph=True)
    penalty = (grad ** 2).sum()  # keeps grad for its backward pass
    version = grad._version
    d2.clip_grads([grad], 1e-3)
    assert grad._version > version
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        penalty.backward()
    # into outputs: these are written, the gradients are not
    g, out = torch.randn(1000, device=DEV), torch.zeros(1000, device=DEV)
    a = torch.ones(1000, device=DEV, requires_grad=True)
    of_g, of_out = (a * g).sum(), (a * out).sum()
    before = g._version
    d2.clip_grads(g, 1e-3, out=out)
    assert g._version == before
    of_g.backward()
    assert torch.equal(a.grad, g)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        of_out.backward()
    before = g._version
    d2.grad_norm(g)
    assert g._version == before


def test_inference_tensors(d2):
    with torch.inference_mode():
        g = torch.full((100,), 2.0, device=DEV)
        norm = d2.clip_grads(g, 1.0)
    assert float(norm) == 20.0 and float((g - 0.1).abs().max()) < 1e-7
    d2.clip_grads(g, 0.5)
    assert float((g - 0.05).abs().max()) < 1e-7
