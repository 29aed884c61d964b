"""The end of a training step with every rank's buffers in one GPU's HBM.

A row-parallel layer leaves N partial results (one per rank) that its norm sums, and
the vocabulary's rows lie in N shards:

    x_r   = a_r p_r                              a product per rank (torch)
    h, y  = layer norm of sum_r x_r + residual   mrr_layernorm_fwd
    loss  = cross entropy of y against all shards' rows     mrr_linear_xent_fwd
    dy, every shard's gradient                   mrr_linear_xent_bwd
    dh, the norm's own gradients                 mrr_layernorm_bwd
    dp_r  = a_r^T dh                             a product per rank (torch)

and all parameters take a step of plain SGD.  The batch is one, drawn at random, so the
loss falls toward zero as it is learnt by heart:

    python examples/training_tail.py --tokens 512 --vocab 8192 --hidden 512 --ranks 4
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import allreduce_reduction_nranks_amd as mrr  # noqa: E402

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
IGNORE = -100
EPS = 1e-5


def shards(vocab, ranks):
    """Rows of each shard: as even as they get, the first ones larger."""
    return [vocab // ranks + (1 if r < vocab % ranks else 0) for r in range(ranks)]


class Tail:
    """Parameters, buffers and workspaces of the tail, allocated once and used by every step.

    The products and buffers are of `dtype`; the parameters are kept in f32 and copied to
    `dtype` after each update, and the loss is scaled where the gradients are f16."""

    def __init__(self, tokens, vocab, hidden, inner, ranks, dtype="bf16", seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        dt = TYPES[dtype]

        def normal(*shape):
            return torch.randn(*shape, generator=g, device="cuda")

        def empty(*shape, dtype=dt):
            return torch.empty(*shape, device="cuda", dtype=dtype)

        self.tokens, self.hidden, self.ranks, self.dtype = tokens, hidden, ranks, dtype
        self.rows = shards(vocab, ranks)
        # what the layers before hand over, and the targets; some tokens have none
        self.acts = [normal(tokens, inner).to(dt) for _ in range(ranks)]
        self.residual = normal(tokens, hidden).to(dt)
        self.targets = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
        self.targets[torch.rand(tokens, generator=g, device="cuda") < 0.1] = IGNORE
        counted = max(1, int((self.targets != IGNORE).sum()))
        # parameters in f32: row-parallel products, the norm's two, the vocabulary's shards
        self.master = ([normal(inner, hidden) / (inner * ranks) ** 0.5 for _ in range(ranks)] +
                       [normal(n, hidden) / hidden ** 0.5 for n in self.rows])
        self.params = [p.to(dt) for p in self.master]
        self.weight, self.bias = torch.ones(hidden, device="cuda"), torch.zeros(hidden, device="cuda")
        # a mean over the counted tokens; f16 gradients are those of a scaled loss
        self.scale = 1024.0 if dtype == "f16" else 1.0
        self.dloss = torch.full((1,), self.scale / counted, device="cuda")
        self.counted = counted
        # results of a step
        self.partial = [empty(tokens, hidden) for _ in range(ranks)]
        self.sum, self.out = empty(tokens, hidden), empty(tokens, hidden)
        self.mean, self.rstd = empty(tokens, dtype=torch.float32), empty(tokens, dtype=torch.float32)
        self.loss, self.lse = empty(tokens, dtype=torch.float32), empty(tokens, dtype=torch.float32)
        self.dout, self.dsum = empty(tokens, hidden), empty(tokens, hidden)
        self.dweight, self.dbias = empty(hidden, dtype=torch.float32), empty(hidden, dtype=torch.float32)
        self.grads = [torch.empty_like(p) for p in self.params]
        # one workspace serves the three calls that need one: they follow each other
        need = max(mrr.mrr_layernorm_bwd_workspace_bytes(tokens, hidden),
                   mrr.mrr_linear_xent_workspace_bytes(tokens, hidden, self.rows, ranks, dtype, False),
                   mrr.mrr_linear_xent_workspace_bytes(tokens, hidden, self.rows, ranks, dtype, True))
        self.workspace = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")

    def gradients(self):
        """Loss and gradients of the present parameters, left in this object's buffers."""
        t, c, n = self.tokens, self.hidden, self.ranks
        shard, ws, wsb = self.params[n:], self.workspace, self.workspace.nbytes
        for r in range(n):
            torch.matmul(self.acts[r], self.params[r], out=self.partial[r])
        mrr.check(mrr.mrr_layernorm_fwd(self.partial, n, self.residual, self.weight, self.bias, self.sum, self.out, self.mean,
                                        self.rstd, t, c, c, c, EPS, self.dtype, "f32"), "layer norm")
        mrr.check(mrr.mrr_linear_xent_fwd(self.out, shard, self.rows, n, self.targets, IGNORE, self.loss, self.lse, t, c, c, c,
                                          self.dtype, ws, wsb), "cross entropy")
        mrr.check(mrr.mrr_linear_xent_bwd(self.out, shard, self.rows, n, self.targets, IGNORE, self.lse, self.dloss, 0,
                                          self.dout, self.grads[n:], t, c, c, c, self.dtype, ws, wsb), "cross entropy gradient")
        mrr.check(mrr.mrr_layernorm_bwd(self.dout, self.sum, self.weight, self.mean, self.rstd, None, self.dsum, self.dweight,
                                        self.dbias, t, c, c, c, self.dtype, "f32", ws, wsb), "layer norm gradient")
        for r in range(n):
            # every rank's partial result has the sum's gradient
            torch.matmul(self.acts[r].t(), self.dsum, out=self.grads[r])

    def update(self, rate):
        for m, p, g in zip(self.master, self.params, self.grads):
            m.sub_(g.float(), alpha=rate / self.scale)
            p.copy_(m)
        self.weight.sub_(self.dweight, alpha=rate / self.scale)
        self.bias.sub_(self.dbias, alpha=rate / self.scale)

    def step(self, rate):
        """One training step; returns the mean loss before it, as a tensor on the GPU."""
        self.gradients()
        self.update(rate)
        return self.loss.sum() / self.counted


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--tokens", type=int, default=512)
    p.add_argument("--vocab", type=int, default=8192)
    p.add_argument("--hidden", type=int, default=512)
    p.add_argument("--inner", type=int, default=256, help="columns of a rank's activations")
    p.add_argument("--ranks", type=int, default=4)
    p.add_argument("--dtype", choices=sorted(TYPES), default="bf16")
    p.add_argument("--steps", type=int, default=20)
    p.add_argument("--rate", type=float, default=8.0)
    p.add_argument("--graph", action="store_true", help="capture a step into a HIP graph and replay it")
    a = p.parse_args(argv)
    tail = Tail(a.tokens, a.vocab, a.hidden, a.inner, a.ranks, a.dtype)
    losses = [tail.step(a.rate).clone()]
    if a.graph:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            tail.gradients()
            tail.update(a.rate)
    for _ in range(a.steps - 1):
        if a.graph:
            graph.replay()
            losses.append(tail.loss.sum() / tail.counted)
        else:
            losses.append(tail.step(a.rate))
    losses = torch.stack(losses).tolist()
    for k, x in enumerate(losses):
        if k % max(1, a.steps // 10) == 0 or k + 1 == a.steps:
            print("step %3d  loss %.4f" % (k, x))
    return losses


if __name__ == "__main__":
    main()
