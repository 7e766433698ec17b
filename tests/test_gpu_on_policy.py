"""Sampling, the top-k pass and the distillation loss together, as a training step on the drafter's own
tokens uses them (needs an MI355X): tokens drawn from the student's logits, the teacher's top logits
after each of them, the loss and its gradient down to the weights.

The student's logits are float32 and their product is torch's; the reference takes the logits as they
are stored, so only this library's kernels and the two products of the backward pass are in the
tolerance: |dz - ref| <= |g| tau (q + 2^-24) eps with eps as in test_gpu_distill, carried through the
products (sums of |dz error| |h| and |W|), plus their fp32 sums, at most (terms + 1) 2^-24 of the sum of
magnitudes.
"""
import math
import sys

import numpy as np
import pytest
import torch

from test_gpu_distill import U, eps_sigma, reference
from test_gpu_sample import f32, reference_row

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def log(*a):
    print(*a, file=sys.stderr, flush=True)


def setup(R, H, V, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)
    hidden = rnd(R, H)
    W = rnd(V, H) * (3.0 / math.sqrt(H))
    teacher = rnd(V, V) * 3.0          # the teacher's logits after each token
    return hidden, W, teacher, g


def step(d2, hidden, W, teacher, uniforms, K, tau):
    """One step: (tokens, logits, ids, unary, loss); gradients land in hidden and W."""
    logits = hidden @ W.t()
    with torch.no_grad():
        tokens, _ = d2.sample(logits, uniforms, temperature=0.9, top_p=0.97)
        ids, unary, _ = d2.topk_lse(teacher[tokens.long()].contiguous(), K)
    loss = d2.distill_loss(logits, ids, unary, tau)
    loss.mean().backward()
    return tokens, logits.detach(), ids, unary, loss.detach()


def test_training_steps():
    import dflash2_draft_candidate_amd as d2
    R, H, V, K, tau = 40, 48, 1501, 12, 1.5
    hidden, W, teacher, g = setup(R, H, V, 4)
    for it in range(3):
        log(f"on-policy step {it}")
        h, w = hidden.clone().requires_grad_(), W.clone().requires_grad_()
        u = torch.rand(R, generator=g, device=DEV)
        tokens, logits, ids, unary, loss = step(d2, h, w, teacher, u, K, tau)
        x = logits.cpu().double().numpy()
        for r in range(R):
            want, _, clear = reference_row(x[r], f32(0.9), 0, f32(0.97), 0.0, float(u[r]))
            assert clear and int(tokens[r]) == want
        rows = teacher[tokens.long()].cpu().double()
        order = torch.from_numpy(np.argsort(-rows.numpy(), axis=1, kind="stable")[:, :K].copy())
        assert torch.equal(ids.cpu().long(), order)
        gl = torch.full((R,), 1.0 / R)
        ref_loss, dz, q = reference(logits, ids, unary, gl, tau)
        assert float((loss.cpu().double() - ref_loss).abs().max()) <= \
            tau * tau * eps_sigma(V) + U * float(ref_loss.abs().max())
        tol_z = (tau / R) * (q + U) * (eps_sigma(V) + 100 * U) + U * dz.abs()
        hd, wd = hidden.cpu().double(), W.cpu().double()
        for got, want, tol, n in (
                (w.grad, dz.t() @ hd,
                 tol_z.t() @ hd.abs() + (R + 1) * U * (dz.abs().t() @ hd.abs()), R),
                (h.grad, dz @ wd, tol_z @ wd.abs() + (V + 1) * U * (dz.abs() @ wd.abs()), V)):
            err = (got.cpu().double() - want).abs()
            assert bool((err <= 1.01 * tol + 1e-12).all()), float((err - tol).max())
        with torch.no_grad():
            W -= 0.5 * w.grad


def test_captured_step():
    """The same step without autograd, captured in a HIP graph and replayed on other inputs."""
    import dflash2_draft_candidate_amd as d2
    R, H, V, K, tau = 32, 32, 2003, 16, 1.0
    hidden, W, teacher, g = setup(R, H, V, 9)
    weights = torch.full((R,), 1.0 / R, device=DEV)

    def run(logits, u):
        tokens, lp = d2.sample(logits, u, temperature=1.1, top_k=50)
        ids, unary, _ = d2.topk_lse(teacher[tokens.long()].contiguous(), K)
        loss, grad = d2.distill_step(logits, ids, unary, weights, tau)
        return tokens, lp, loss, grad

    inputs = []
    for _ in range(3):
        inputs.append(((torch.randn(R, H, generator=g, device=DEV) @ W.t()).contiguous(),
                       torch.rand(R, generator=g, device=DEV)))
    buf = [t.clone() for t in inputs[0]]
    run(*buf)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(*buf)
    for logits, u in inputs + inputs[:1]:
        buf[0].copy_(logits)
        buf[1].copy_(u)
        graph.replay()
        torch.cuda.synchronize()
        want = run(logits, u)
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)
