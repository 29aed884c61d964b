"""The example that runs layer norm, cross entropy and both gradients as one training
step: its gradients against autograd of the whole step in 64 bits, and its loss.

f32: each of at most 6 stages in a row is off by at most 2^-24 times its count of terms
(under 4096 here), relative to its terms' sizes.  16-bit types: a gradient passes 5
roundings (partial result, sum, norm, dy, its own) of half a step, each relative to
elements within 8 of the largest."""
import importlib.util
import os

import pytest
import torch

from gpu_common import announce

pytestmark = pytest.mark.gpu

spec = importlib.util.spec_from_file_location(
    "training_tail", os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "training_tail.py"))
example = importlib.util.module_from_spec(spec)
spec.loader.exec_module(example)

TOL = {"f32": 6 * 4096 * 2.0 ** -24, "f16": 8 * 5 * 2.0 ** -11, "bf16": 8 * 5 * 2.0 ** -8}


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("tokens,vocab,hidden,inner,ranks", [(3, 50, 40, 16, 2), (130, 1003, 192, 64, 3), (257, 2048, 256, 32, 8)])
def test_gradients_of_the_whole_step(tokens, vocab, hidden, inner, ranks, t):
    announce("training tail", t, tokens, vocab, hidden, ranks)
    tail = example.Tail(tokens, vocab, hidden, inner, ranks, t, seed=tokens)
    tail.gradients()
    torch.cuda.synchronize()
    leaf = [p.detach().double().cpu().requires_grad_() for p in tail.params + [tail.weight, tail.bias]]
    x = tail.residual.double().cpu() + sum(a.double().cpu() @ p for a, p in zip(tail.acts, leaf))
    xhat = (x - x.mean(1, keepdim=True)) / torch.sqrt(x.var(1, unbiased=False, keepdim=True) + example.EPS)
    y = xhat * leaf[-2] + leaf[-1]
    z = y @ torch.cat(leaf[ranks:-2]).T
    loss = torch.nn.functional.cross_entropy(z, tail.targets.cpu(), ignore_index=example.IGNORE, reduction="none")
    (loss.sum() * float(tail.dloss[0])).backward()
    tol = TOL[t]
    assert float((tail.loss.double().cpu() - loss.detach()).abs().max()) <= tol * float(z.detach().abs().max())
    for k, (got, want) in enumerate(zip(tail.grads + [tail.dweight, tail.dbias], leaf)):
        assert float((got.double().cpu() - want.grad).abs().max()) <= tol * float(want.grad.abs().max()), k


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
def test_the_batch_is_learnt(t, graph):
    announce("training tail learns", t, graph)
    args = ["--tokens", "100", "--vocab", "1000", "--hidden", "128", "--inner", "64", "--ranks", "4", "--dtype", t, "--steps", "12"]
    losses = example.main(args + (["--graph"] if graph else []))
    assert losses[0] > 5.0 and losses[-1] < 0.5 * losses[0]
