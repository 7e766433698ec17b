"""Per-row numbers that are slices of a batch's tensors, off the 16 bytes that the library asks of a
pointer (needs an MI355X): the same results as from copies, bit for bit, and outputs land in the slices
and nowhere else. Logits and gradients have to start on 16 bytes: slices that do not are refused."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def d2():
    import dflash2_draft_candidate_amd
    return dflash2_draft_candidate_amd


def off(t, by=1):
    """The same values, starting `by` elements into a larger tensor."""
    whole = torch.empty(by + t.numel(), dtype=t.dtype, device=t.device)
    whole[by:] = t.flatten()
    s = whole[by:].view(t.shape)
    assert s.data_ptr() % 16 != 0
    return s


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,V", [(5, 4096), (6, 90000)])
def test_sample(d2, R, V, dtype):
    g = torch.Generator(device=DEV).manual_seed(V)
    x = (torch.randn(R, V, generator=g, device=DEV) * 3).to(dtype)
    u = torch.rand(R, generator=g, device=DEV)
    t = torch.tensor([0.0, 0.7, 1.0, 1.3, 0.9, 2.0], device=DEV)[:R].clone()
    k = torch.tensor([0, 5, 40, 0, 3000, 1], dtype=torch.int32, device=DEV)[:R].clone()
    p = torch.tensor([1.0, 0.9, 0.95, 0.5, 1.0, 0.99], device=DEV)[:R].clone()
    m = torch.tensor([0.0, 0.1, 0.0, 0.02, 0.0, 0.0], device=DEV)[:R].clone()
    want = d2.sample(x, u, t, k, p, m)
    for by in (1, 2, 3):
        got = d2.sample(x, off(u, by), off(t, by), off(k, by), off(p, by), off(m, by))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        ids = torch.full((R + 8,), -7, dtype=torch.int32, device=DEV)
        lp = torch.full((R + 8,), 7.0, device=DEV)
        out = (ids[by:by + R], lp[by:by + R])
        got = d2.sample(x, off(u, by), off(t, by), k, p, off(m, by), out=out)
        assert got[0] is out[0] and got[1] is out[1]
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
        for whole, fill in ((ids, -7), (lp, 7.0)):
            assert bool((whole[:by] == fill).all()) and bool((whole[by + R:] == fill).all())
    # two rows of a batch, as a program that serves them apart takes them
    rows = (x[2:4], u[2:4], t[2:4], k[2:4], p[2:4], m[2:4])
    got, want = d2.sample(*rows), d2.sample(*(a.clone() for a in rows))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(d2.Dflash2Error):
        d2.sample(off(x), u)


def test_sample_captured(d2):
    R, V = 7, 3000
    x = torch.randn(R, V, device=DEV)
    u, t = off(torch.rand(R, device=DEV)), off(torch.full((R,), 0.8, device=DEV))
    ids, lp = off(torch.zeros(R, dtype=torch.int32, device=DEV)), off(torch.zeros(R, device=DEV))
    d2.sample(x, u, t, out=(ids, lp))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d2.sample(x, u, t, out=(ids, lp))
    for _ in range(4):
        u.copy_(torch.rand(R, device=DEV))
        t.copy_(torch.rand(R, device=DEV) + 0.5)
        graph.replay()
        torch.cuda.synchronize()
        want = d2.sample(x, u.clone(), t.clone())
        torch.cuda.synchronize()
        assert torch.equal(ids, want[0]) and torch.equal(lp, want[1])


@pytest.mark.parametrize("R,V,K", [(9, 4096, 7), (16, 165000, 5), (130, 20000, 3)])
def test_distill(d2, R, V, K):
    g = torch.Generator(device=DEV).manual_seed(V)
    z = (torch.randn(R, V, generator=g, device=DEV) * 3).bfloat16()
    ids = torch.randint(-1, V, (R, K), generator=g, device=DEV, dtype=torch.int32)
    t = torch.randn(R, K, generator=g, device=DEV)
    gl = torch.rand(R, generator=g, device=DEV)
    loss, stats = d2.distill(z, ids, t, 1.5)
    grad = d2.distill_backward(z, ids, t, stats, gl, 1.5)
    step = d2.distill_step(z, ids, t, gl, 1.5)
    a = d2.distill(z, off(ids), off(t), 1.5)
    assert torch.equal(a[0], loss) and torch.equal(a[1], stats)
    assert torch.equal(d2.distill_backward(z, off(ids), off(t, 3), off(stats, 2), off(gl), 1.5), grad)
    b = d2.distill_step(z, off(ids, 2), off(t), off(gl, 3), 1.5)
    assert torch.equal(b[0], step[0]) and torch.equal(b[1], step[1])
    # rows of a batch, under autograd
    results = []
    for rows in ((ids[1:], t[1:], gl[1:]), (ids[1:].clone(), t[1:].clone(), gl[1:].clone())):
        zr = z[1:].clone().requires_grad_()
        loss = d2.distill_loss(zr, rows[0], rows[1], 1.5)
        loss.backward(rows[2])
        results.append((loss.detach(), zr.grad))
    assert torch.equal(results[0][0], results[1][0]) and torch.equal(results[0][1], results[1][1])
    with pytest.raises(d2.Dflash2Error):
        d2.distill(off(z), ids, t, 1.5)
    with pytest.raises(d2.Dflash2Error):
        d2.distill_step(z, ids, t, gl, 1.5, out=off(torch.zeros_like(z)))
