"""GPU checks of f32 cross entropy calls whose rows differ by many orders of magnitude: a
row's error depends on that row alone, not on the largest value of a tensor, whichever way
a call's size makes it multiply.

Tolerances, with u = 2^-24:
- a logit is a sum of C products.  As f32 products each adds u of itself and of the sum so
  far; as 6 products of bf16 parts, what is left out is 2^-26 of each, the five smaller ones
  are below 2^-7 of the whole together, and so are their roundings.  A matrix instruction's
  own additions are given a whole step, 2 u, each: (2.2 C + 8) u of the sum of sizes;
- lse moves by the logits' errors weighted with p, by the chain of its sum and by its own
  rounding; the loss by that, the target logit's error and its own rounding;
- p is off by what the logit's error and the rounding of z - lse make of it and by 4 u for
  the exponential and two products; p - 1 by its rounding as well;
- a gradient is off by its terms' errors, by (2.2 n + 64) u of its n terms' sizes, and by u
  for its rounding.
"""
import pytest
import torch

import allreduce_reduction_nranks_amd as mrr
from gpu_common import announce

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
IGNORE = -100


def seeded(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def close(got, want, tol, what):
    off = (got.double() - want).abs()
    bad = ~(off <= tol)
    assert not bool(bad.any()), "%s: %d of %d off, worst %.3g of the tolerance" % (
        what, int(bad.sum()), bad.numel(), float((off / tol.clamp(min=1e-300)).max()))


class Call:
    def __init__(self, tokens, rows, cols, seed):
        g = self.g = seeded(seed)
        self.tokens, self.rows, self.cols = tokens, rows, cols
        self.hidden = torch.randn(tokens, cols, generator=g, device="cuda")
        self.weights = [torch.randn(n, cols, generator=g, device="cuda") / cols ** 0.5 for n in rows]
        self.targets = torch.randint(0, sum(rows), (tokens,), generator=g, device="cuda")
        self.dloss = 0.5 + torch.rand(tokens, generator=g, device="cuda")

    def uniform(self, n):
        return torch.rand(n, generator=self.g, device="cuda")

    def workspace(self, backward):
        n = mrr.mrr_linear_xent_workspace_bytes(self.tokens, self.cols, self.rows, len(self.rows), "f32", backward)
        return torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device="cuda"), n

    def forward(self):
        loss, lse = torch.empty(self.tokens, device="cuda"), torch.empty(self.tokens, device="cuda")
        ws, n = self.workspace(False)
        mrr.check(mrr.mrr_linear_xent_fwd(self.hidden, self.weights, self.rows, len(self.rows), self.targets, IGNORE, loss, lse,
                                          self.tokens, self.cols, self.cols, self.cols, "f32", ws, n))
        return loss, lse

    def backward(self, lse):
        dh, dw = torch.empty_like(self.hidden), [torch.empty_like(w) for w in self.weights]
        ws, n = self.workspace(True)
        mrr.check(mrr.mrr_linear_xent_bwd(self.hidden, self.weights, self.rows, len(self.rows), self.targets, IGNORE, lse,
                                          self.dloss, 1, dh, dw, self.tokens, self.cols, self.cols, self.cols, "f32", ws, n))
        return dh, dw

    def logits(self):
        h, w = self.hidden.double(), torch.cat(self.weights).double()
        return h, w, h @ w.T, (2.2 * self.cols + 8) * U * (h.abs() @ w.abs().T)

    def check_forward(self, tokens=slice(None)):
        """Of the tokens given: the others' own loss says nothing."""
        loss, lse = self.forward()
        h, w, z, ez = (x if i == 1 else x[tokens] for i, x in enumerate(self.logits()))
        want = torch.logsumexp(z, 1)
        p = (z - want[:, None]).exp()
        size = (p * z.abs()).sum(1) + z.abs().amax(1)
        tol = (p * ez).sum(1) * 1.01 + U * (4 * size + 256 + z.shape[1] / 4096 + 4 * want.abs()) + ez.amax(1) ** 2
        close(lse[tokens], want, tol, "lse")
        at = self.targets[tokens].clamp(min=0)[:, None]
        zt, ezt = z.gather(1, at)[:, 0], ez.gather(1, at)[:, 0]
        counted = self.targets[tokens] != IGNORE
        close(loss[tokens], torch.where(counted, want - zt, 0.0), torch.where(counted, tol + ezt + U * (want - zt).abs(), 0.0), "loss")

    def check_backward(self):
        h, w, z, ez = self.logits()
        lse = torch.logsumexp(z, 1).float()
        dh, dw = self.backward(lse)
        x = z - lse.double()[:, None]
        p = x.exp()
        counted = self.targets != IGNORE
        dl = torch.where(counted, self.dloss.double(), 0.0)[:, None]
        hit = torch.zeros_like(p).scatter_(1, self.targets.clamp(min=0)[:, None], 1.0)
        dz = (p - hit) * dl
        edz = (p * (torch.expm1(ez + U * x.abs()) + 4 * U) + 2 * U * hit) * dl.abs()

        def grad(a, ea, b, terms, got, what):
            want = a @ b
            tol = ea @ b.abs() + (2.2 * terms + 64) * U * ((a.abs() + ea) @ b.abs()) + U * want.abs()
            close(got, want, tol * 1.01, what)

        grad(dz, edz, w, w.shape[0], dh, "dhidden")
        grad(dz.T.contiguous(), edz.T.contiguous(), torch.where(counted[:, None], h, 0.0), self.tokens, torch.cat(dw), "dweights")


#: few products (multiplied as f32), and many (as parts)
SIZES = [(5, [300, 41], 64), (300, [400, 111], 72), (2000, [30000], 128)]


@pytest.mark.parametrize("tokens,rows,cols", SIZES)
def test_an_ignored_token_s_hidden_state_does_not_reach_the_others_loss(tokens, rows, cols):
    announce("xent spread ignored", tokens, rows, cols)
    c = Call(tokens, rows, cols, 1)
    c.targets[1] = IGNORE
    c.hidden[1] *= 1e30
    c.check_forward(torch.arange(tokens, device="cuda") != 1)


@pytest.mark.parametrize("tokens,rows,cols", SIZES)
def test_a_large_weight_that_no_token_reads(tokens, rows, cols):
    announce("xent spread weight", tokens, rows, cols)
    c = Call(tokens, rows, cols, 2)
    c.hidden[:, 0] = 0.0
    c.weights[0][5, 0] = 1e12
    c.check_forward()
    if tokens <= 300:
        c.check_backward()


@pytest.mark.parametrize("tokens,rows,cols", SIZES[:2] + [(1000, [2000, 777], 96)])
def test_loss_gradients_nine_orders_apart(tokens, rows, cols):
    announce("xent spread dloss", tokens, rows, cols)
    c = Call(tokens, rows, cols, 3)
    c.dloss = 10.0 ** (-9 * c.uniform(tokens))
    c.check_backward()


@pytest.mark.parametrize("tokens,rows,cols", SIZES[:2] + [(1000, [2000, 777], 96)])
def test_hidden_states_nine_orders_apart_in_a_column_without_weights(tokens, rows, cols):
    """Each token's share of that column's gradient is of one size, as its loss gradient
    makes up for its hidden state."""
    announce("xent spread hidden", tokens, rows, cols)
    c = Call(tokens, rows, cols, 4)
    c.hidden[:, 0] = 10.0 ** (9 * c.uniform(tokens))
    for w in c.weights:
        w[:, 0] = 0.0
    c.dloss = c.dloss / c.hidden[:, 0]
    c.check_backward()


@pytest.mark.parametrize("scale", [1e-30, 1e30])
def test_weights_and_hidden_states_near_the_ends_of_f32(scale):
    """Logits of ordinary size from operands that are not."""
    announce("xent spread ends", scale)
    c = Call(300, [400, 111], 72, 5)
    c.hidden *= scale
    for w in c.weights:
        w /= scale
    c.check_forward()
    c.check_backward()
