"""The few-row top-k pass on workspaces that hold other data (needs an MI355X).

A workspace need not be initialised: whatever it holds before a call, the outputs are those of a
zeroed one, bit for bit. What it holds here, per 64-bit word, are numbers that count up in the upper half
(from 0, from 0x7FB10000, bf16 pairs of NaN and of -0, -0.0f) above small counts, another run of 64 at
each call; eager, and before each replay of a graph.
"""
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
UPPER = [0, 0x7FB10000, 0x7FC00000, 0x80000000, 0xFFC00000]


def log(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module")
def d2():
    import dflash2_draft_candidate_amd
    return dflash2_draft_candidate_amd


class Pass:
    def __init__(self, d2, R, V, k, dtype, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.lib, self.k, self.dt = d2.library(), k, 0 if dtype == torch.float32 else 1
        self.x = (torch.randn(R, V, generator=g, device=DEV) * 3).to(dtype)
        nbytes = self.lib.dflash2_topk_lse_workspace_bytes(R, V, k, self.dt)
        assert nbytes > 0  # (rows in slices)
        self.ws = torch.zeros((nbytes + 15) // 16 * 2, dtype=torch.int64, device=DEV)
        self.out = (torch.empty(R, k, dtype=torch.int32, device=DEV),
                    torch.empty(R, k, dtype=torch.float32, device=DEV),
                    torch.empty(R, dtype=torch.float32, device=DEV))

    def clear(self):
        for t in self.out:
            t.fill_(-7)

    def launch(self):
        R, V = self.x.shape
        p = [t.data_ptr() for t in self.out]
        assert self.lib.dflash2_topk_lse(self.x.data_ptr(), self.dt, R, V, self.k, *p,
                                         self.ws.data_ptr(), self.ws.numel() * 8,
                                         torch.cuda.current_stream().cuda_stream) == 0


def words(n, upper, first, count):
    w = torch.arange(n, device=DEV, dtype=torch.int64) % 64 + (first % 1024 + upper)
    w = torch.where(w >= 2 ** 31, w - 2 ** 32, w)
    return (w << 32) + count


SHAPES = [(64, 20000, 8, torch.bfloat16), (16, 151936, 16, torch.bfloat16), (1, 100003, 64, torch.float32),
          (40, 9001, 5, torch.float32)]


@pytest.mark.parametrize("R,V,k,dtype", SHAPES)
def test_any_contents(d2, R, V, k, dtype):
    log(f"few-row pass, workspace contents R={R} V={V} k={k} {dtype}")
    a = Pass(d2, R, V, k, dtype, R + V)
    a.launch()
    want = [t.clone() for t in a.out]
    n = a.ws.numel()
    bad = torch.zeros((), dtype=torch.int64, device=DEV)
    for call in range(400):
        for upper in UPPER[:2] if call % 16 else UPPER:
            a.ws.copy_(words(n, upper, call * 64, 1 + call % 5))
            a.clear()
            a.launch()
            for t, w in zip(a.out, want):
                bad += (t != w).sum()
    assert int(bad) == 0


@pytest.mark.parametrize("R,V,k,dtype", SHAPES)
def test_any_contents_before_a_replay(d2, R, V, k, dtype):
    a = Pass(d2, R, V, k, dtype, R * 3 + V)
    a.launch()
    torch.cuda.synchronize()
    want = [t.clone() for t in a.out]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.launch()
    n = a.ws.numel()
    for call in range(60):
        a.ws.copy_(words(n, UPPER[call % len(UPPER)], call * 64, call % 9))
        a.clear()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t, w) for t, w in zip(a.out, want))
        if call % 7 == 0:  # an eager call on the same workspace in between
            a.clear()
            a.launch()
            torch.cuda.synchronize()
            assert all(torch.equal(t, w) for t, w in zip(a.out, want))
