"""GPU check of cross entropy gradients of up to 64 tokens in 16 bits: their error is that of their
own rounding, whichever way the logits are computed."""
import pytest
import torch

import allreduce_reduction_nranks_amd as mrr
from gpu_common import announce
from xent_few_tokens import Few

pytestmark = pytest.mark.gpu


def run(c, dhidden=True, dweights=True):
    rows = c.rows
    like = lambda x: torch.full((x.shape[0], c.ld), 7.0, dtype=x.dtype, device="cuda")[:, :c.cols]  # noqa: E731
    dh = like(c.hidden) if dhidden else None
    dw = [like(w) for w in c.weights] if dweights else None
    n = mrr.mrr_linear_xent_workspace_bytes(c.tokens, c.cols, rows, len(rows), c.t, True)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    mrr.check(mrr.mrr_linear_xent_bwd(c.hidden, c.weights, rows, len(rows), c.targets, -100, c.lse, c.dloss, 1, dh, dw, c.tokens,
                                      c.cols, c.ld, c.ld, c.t, ws, n))
    torch.cuda.synchronize()
    return dh, dw


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("tokens,rows,cols,pad", [
    (1, [300, 600], 128, 0), (2, [40, 1], 64, 0), (4, [300, 600], 130, 1), (5, [2000, 1000], 1024, 0), (17, [300, 600], 130, 0),
    (32, [300, 600], 128, 0), (31, [5, 600], 65, 0), (33, [700, 0, 300], 192, 8), (63, [300, 600], 128, 0), (64, [300, 600], 257, 3), (64, [3000, 1000], 512, 0),
])
def test_gradients_have_their_own_rounding_alone(tokens, rows, cols, pad, t):
    announce("xent few tokens", t, tokens, rows, cols, pad)
    c = Few(tokens, rows, cols, t, tokens + cols, "cuda", pad=pad)
    dh, dw = run(c)
    assert c.off(dh, torch.cat(dw)) == [0, 0]
    for x in [dh] + dw:
        if pad and len(x):  # nothing beside the rows is written
            assert bool((x.as_strided((len(x), pad), (c.ld, 1), cols) == 7).all())


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("tokens,ignored", [(1, 1), (9, 3), (32, 5), (33, 1), (64, 1), (64, 63), (40, 40)])
def test_tokens_without_a_loss_among_them(tokens, ignored, t):
    announce("xent few tokens ignored", t, tokens, ignored)
    c = Few(tokens, [300, 600], 192, t, tokens + ignored, "cuda", ignored=ignored)
    c.hidden[:ignored] = float("nan")
    c.h = torch.where(c.targets[:, None] >= 0, c.hidden.double(), 0.0)
    c.dz, c.edz = (torch.where(c.targets[:, None] >= 0, x, 0.0) for x in (c.dz, c.edz))
    dh, dw = run(c)
    assert c.off(dh, torch.cat(dw)) == [0, 0]
    assert not bool(dh[:ignored].any())


@pytest.mark.parametrize("tokens", [3, 50])
def test_weights_that_are_infinite_stay_with_their_tokens(tokens):
    """A row of -inf weights against positive hidden states has probability 0: no other row's
    gradient sees it, whatever stands in the places of tokens that are not there."""
    announce("xent few tokens inf", tokens)
    c = Few(tokens, [300, 600], 128, "bf16", 3, "cuda")
    c.hidden.abs_().add_(0.1)
    c.weights[1][7] = -float("inf")
    z = c.hidden.double() @ torch.cat(c.weights).double().T
    c.lse = torch.logsumexp(z, 1).float()
    dh, dw = run(c, dhidden=False)
    assert all(bool(w.isfinite().all()) for w in dw) and not bool(dw[1][7].any())


@pytest.mark.parametrize("tokens", [4, 64])
def test_each_gradient_alone_is_the_same(tokens):
    announce("xent few tokens alone", tokens)
    c = Few(tokens, [300, 600], 128, "bf16", 5, "cuda")
    dh, dw = run(c)
    assert torch.equal(run(c, dweights=False)[0], dh)
    assert all(torch.equal(a, b) for a, b in zip(run(c, dhidden=False)[1], dw))
