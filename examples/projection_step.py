"""A training step of a projection to queries, keys and values on N data-parallel ranks, with
every rank's buffers in one GPU's HBM.

Each rank has tokens of its own and a copy of the weights, which lie in `parts` row-parallel
pieces:

    x_p      = a_p W_p                                a product per piece (torch)
    h, q, k, v = sum_p x_p, its head norms and rotation     mrr_qknorm_rope_fwd
    dq, dk, dv = those of half the squared distance to targets, which stand for attention
    dh, the norms' own gradients                      mrr_qknorm_rope_bwd
    dW_p     = a_p^T dh                               a product per piece (torch)

and one call sums the ranks' gradients and updates every rank's weights (mrr_muon_step, the
pieces as its batch); the norms' two vectors take a step of plain SGD.

    python examples/projection_step.py --tokens 512 --heads 8 2 2 --dim 64 --ranks 4
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import allreduce_reduction_nranks_amd as mrr  # noqa: E402

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6
STEPS = 5


def rotation_table(rows, rot, base=10000.0):
    """Cosines, then sines, of each position's angles, computed in 64 bits."""
    half = rot // 2
    f = base ** (-torch.arange(half, device="cuda", dtype=torch.float64) / max(1, half))
    a = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


class Rank:
    """One data-parallel rank's tokens and buffers."""

    def __init__(self, g, tokens, heads, dim, inner, parts, dt):
        width = sum(heads) * dim
        self.acts = torch.randn(parts, tokens, inner, generator=g, device="cuda").to(dt)
        # two sequences side by side; the last tokens of the second fill up the batch
        t = torch.arange(tokens, device="cuda")
        self.positions = torch.where(t < tokens // 2, t, t - tokens // 2)
        self.positions[tokens - tokens // 8:] = -1
        self.targets = [torch.randn(tokens, n, dim, generator=g, device="cuda").to(dt) for n in heads]
        self.partial = torch.empty(parts, tokens, width, device="cuda", dtype=dt)
        self.sum = torch.zeros(tokens, width, device="cuda", dtype=dt)
        self.outs = [torch.zeros(tokens, n, dim, device="cuda", dtype=dt) for n in heads]
        self.douts = [torch.zeros_like(o) for o in self.outs]
        self.dsum = torch.empty_like(self.sum)
        self.dnorm = torch.empty(2, dim, device="cuda")
        self.grad = torch.empty(parts, inner, width, device="cuda", dtype=dt)


class Step:
    """Weights, momentum and buffers of all ranks, allocated once and used by every step.  Products
    and buffers are of `dtype`, the momentum and the norms' weights of f32."""

    def __init__(self, tokens, heads, dim, rot, inner, parts, ranks, dtype="bf16", seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        dt = TYPES[dtype]
        self.tokens, self.heads, self.dim, self.rot, self.inner, self.dtype = tokens, list(heads), dim, rot, inner, dtype
        self.width, self.parts = sum(heads) * dim, parts
        self.table = rotation_table(tokens, rot)
        self.norm = torch.ones(2, dim, device="cuda")  # of the queries and keys
        w = torch.randn(parts, inner, self.width, generator=g, device="cuda") / (parts * inner) ** 0.5
        self.weights = [w.to(dt, copy=True) for _ in range(ranks)]
        self.momentum = torch.zeros(parts, inner, self.width, device="cuda")
        self.ranks = [Rank(g, tokens, self.heads, dim, inner, parts, dt) for _ in range(ranks)]
        # one workspace serves both calls that need one: they follow each other
        need = max(mrr.mrr_qknorm_rope_bwd_workspace_bytes(tokens, self.heads, dim),
                   mrr.mrr_muon_workspace_bytes(inner, self.width, parts, dtype))
        self.workspace = torch.empty(need, dtype=torch.uint8, device="cuda")

    def gradients(self):
        """Outputs and gradients of the present weights, left in the ranks' buffers."""
        lds, strides, ws = [n * self.dim for n in self.heads], [self.dim] * 3, self.workspace
        for r, w in zip(self.ranks, self.weights):
            for p in range(self.parts):
                torch.matmul(r.acts[p], w[p], out=r.partial[p])
            mrr.check(mrr.mrr_qknorm_rope_fwd(list(r.partial), self.parts, self.norm[0], self.norm[1], self.table, self.tokens,
                                              r.positions, r.sum, r.outs, self.tokens, self.heads, self.dim, self.rot, False, self.width,
                                              lds, strides, EPS, self.dtype, "f32"), "head norms")
            for d, o, t in zip(r.douts, r.outs, r.targets):
                torch.sub(o, t, out=d)
            mrr.check(mrr.mrr_qknorm_rope_bwd(r.douts, r.sum, self.norm[0], self.norm[1], self.table, self.tokens, r.positions,
                                              r.dsum, r.dnorm[0], r.dnorm[1], self.tokens, self.heads, self.dim, self.rot, False,
                                              self.width, lds, strides, EPS, self.dtype, "f32", ws, ws.nbytes), "head norms' gradient")
            for p in range(self.parts):
                # every piece's partial result has the sum's gradient
                torch.matmul(r.acts[p].t(), r.dsum, out=r.grad[p])

    def update(self, rate, mu=0.9, decay=0.0):
        n, per = len(self.ranks), self.inner * self.width
        mrr.check(mrr.mrr_muon_step([r.grad for r in self.ranks], n, 1.0 / n, self.momentum, self.momentum, mu, True, self.weights[0],
                                    self.weights, rate, decay, self.inner, self.width, self.width, self.width, self.parts, per, per, STEPS,
                                    None, 1e-7, self.dtype, self.dtype, "auto", self.workspace, self.workspace.nbytes), "update")
        for r in self.ranks:
            self.norm.sub_(r.dnorm, alpha=rate / (n * self.tokens * self.dim))

    def loss(self):
        """Half the squared distance to the targets, a value of the tokens that count, as a tensor on the GPU."""
        total = sum((d.float().square() * (r.positions >= 0)[:, None, None]).sum() for r in self.ranks for d in r.douts)
        return total / (2 * len(self.ranks) * self.tokens * self.width)


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--tokens", type=int, default=512, help="of a rank")
    p.add_argument("--heads", type=int, nargs=3, default=[8, 2, 2], help="of the queries, keys and values")
    p.add_argument("--dim", type=int, default=64, help="of a head")
    p.add_argument("--rot", type=int, default=None, help="rotated elements of a head (all)")
    p.add_argument("--inner", type=int, default=256, help="rows of a piece of the weights")
    p.add_argument("--parts", type=int, default=2)
    p.add_argument("--ranks", type=int, default=4)
    p.add_argument("--dtype", choices=sorted(TYPES), default="bf16")
    p.add_argument("--steps", type=int, default=20)
    p.add_argument("--rate", type=float, default=0.05)
    p.add_argument("--graph", action="store_true", help="capture a step into a HIP graph and replay it")
    a = p.parse_args(argv)
    s = Step(a.tokens, a.heads, a.dim, a.dim if a.rot is None else a.rot, a.inner, a.parts, a.ranks, a.dtype)

    def one():
        s.gradients()
        s.update(a.rate)

    one()
    losses, graph = [s.loss()], None
    if a.graph:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            one()
    for _ in range(a.steps - 1):
        graph.replay() if graph else one()
        losses.append(s.loss())
    losses = torch.stack(losses).tolist()
    for k, x in enumerate(losses):
        if k % max(1, a.steps // 10) == 0 or k + 1 == a.steps:
            print("step %3d  loss %.4f" % (k, x))
    return losses


if __name__ == "__main__":
    main()
