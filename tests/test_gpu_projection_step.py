"""The example that runs head norms with rotation, their gradient and the weights' update as one
training step of several ranks: its gradients against autograd of the whole step in 64 bits,
its update against the formula on its own gradients, and a captured step against eager ones.

Gradients, f32: each of at most 5 stages in a row is off by at most 2^-24 times its count of terms
(under 4096 here), relative to its terms' sizes.  16-bit types: a gradient passes 5 roundings
(partial result, sum, output, difference, its own) of half a step and that of dh, each relative
to elements within 8 of the largest.  The update: results of the products are off by up to 4e-3 of
their norm in 16 bits (their own bounds are tested apart) and 1e-5 in 32, and the weights round once."""
import importlib.util
import os

import pytest
import torch

from gpu_common import announce

pytestmark = pytest.mark.gpu

spec = importlib.util.spec_from_file_location(
    "projection_step", os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "projection_step.py"))
example = importlib.util.module_from_spec(spec)
spec.loader.exec_module(example)

TOL = {"f32": 5 * 4096 * 2.0 ** -24, "f16": 8 * 6 * 2.0 ** -11, "bf16": 8 * 6 * 2.0 ** -8}
CO = (3.4445, -4.7750, 2.0315)


def whole_step(rank, w, norm, table, heads, dim, rot):
    """Half the squared distance to the targets, in 64 bits on the CPU."""
    h = sum(rank.acts[p].double().cpu() @ w[p] for p in range(len(w)))
    pos = rank.positions.cpu()
    row = table.double().cpu()[pos.clamp(min=0)][:, None]
    c, s = row[..., :rot // 2], row[..., rot // 2:]
    total, first = 0.0, 0
    for k, n in enumerate(heads):
        x = h[:, first * dim:(first + n) * dim].reshape(len(h), n, dim)
        first += n
        if k < 2:
            x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + example.EPS) * norm[k]
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            x = torch.cat([a * c - b * s, b * c + a * s, x[..., rot:]], -1)
        total = total + ((x - rank.targets[k].double().cpu()).square() * (pos >= 0)[:, None, None]).sum() / 2
    return total


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("tokens,heads,dim,rot,inner,parts,ranks", [(24, (2, 1, 1), 16, 16, 40, 1, 2), (130, (4, 2, 1), 48, 24, 96, 3, 2)])
def test_gradients_and_update_of_the_whole_step(tokens, heads, dim, rot, inner, parts, ranks, t):
    announce("projection step", t, tokens, heads, dim, parts, ranks)
    s = example.Step(tokens, heads, dim, rot, inner, parts, ranks, t, seed=tokens)
    s.norm.mul_(1.0 + 0.2 * torch.randn_like(s.norm))
    s.gradients()
    torch.cuda.synchronize()
    for rank, weight in zip(s.ranks, s.weights):
        w = weight.double().cpu().requires_grad_()
        norm = s.norm.double().cpu().requires_grad_()
        whole_step(rank, w, norm, s.table, heads, dim, rot).backward()
        for got, want in ((rank.grad, w.grad), (rank.dnorm, norm.grad)):
            assert float((got.double().cpu() - want).abs().max()) <= TOL[t] * float(want.abs().max())
    before = s.weights[0].double()
    g = sum(r.grad.double() for r in s.ranks) / ranks
    s.update(0.05, mu=0.9, decay=0.01)
    torch.cuda.synchronize()
    assert all(torch.equal(x, s.weights[0]) for x in s.weights)
    assert float((s.momentum.double() - g).norm()) <= 2.0 ** -22 * float(g.norm())
    for p in range(parts):
        x = g[p] * 1.9
        x = x / (x.norm() + 1e-7)
        turn = x.shape[0] > x.shape[1]
        x = x.T.contiguous() if turn else x
        for _ in range(5):
            m = x @ x.T.contiguous()
            x = CO[0] * x + (CO[1] * m + CO[2] * m @ m) @ x
        x = x.T if turn else x
        want = 0.99 * before[p] - 0.05 * x
        off = float((s.weights[0][p].double() - want).norm())
        assert off <= (torch.finfo(example.TYPES[t]).eps / 2) * float(want.norm()) + 0.05 * (1e-5 if t == "f32" else 4e-3) * float(x.norm())


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_a_captured_step_is_the_eager_one(t):
    announce("projection step graph", t)
    args = ["--tokens", "100", "--heads", "4", "2", "2", "--dim", "32", "--inner", "48", "--ranks", "3", "--dtype", t, "--steps", "5"]
    losses = example.main(args)
    assert len(losses) == 5 and all(0.0 < x < 1e6 for x in losses)
    assert example.main(args + ["--graph"]) == losses
