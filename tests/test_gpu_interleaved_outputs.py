"""GPU checks of outputs that lie between each other: heads of the queries, keys and values in turn in one buffer, of the head
norms and of the gradients that their backward reads; weights and momenta as column slices of one buffer.  A result must be
bit for bit that of separate buffers."""
import pytest
import torch

import allreduce_reduction_nranks_amd as mrr
from gpu_common import announce
from test_gpu_muon import gradient, muon
from test_gpu_qknorm import TYPES, backward, empty_outs, forward, randn, seeded, table_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,n,dim,rot", [(1, 4, 64, 64), (37, 3, 41, 20), (50, 5, 80, 32)])
@pytest.mark.parametrize("way", ["tokens", "heads"])
def test_heads_in_turn(t, tokens, n, dim, rot, way):
    announce("qk in turn", t, tokens, n, dim, rot, way)
    g = seeded(tokens + dim)
    heads, width = [n] * 3, 3 * n * dim
    inputs = [randn(g, tokens, width, t=t) for _ in range(2)]
    table, weights = table_of(rot), [randn(g, dim), randn(g, dim)]
    want, total, dsum = empty_outs(tokens, heads, dim, t), torch.empty_like(inputs[0]), torch.empty_like(inputs[0])
    mrr.check(forward(inputs, weights, table, None, total, want, heads, dim, rot, False, t, "f32"))
    if way == "tokens":
        buffer = torch.full((tokens, n, 3, dim), 7.0, dtype=TYPES[t], device="cuda")
        outs, lds, strides = [buffer[:, :, k] for k in range(3)], [width] * 3, [3 * dim] * 3
    else:
        buffer = torch.full((n, tokens, 3, dim), 7.0, dtype=TYPES[t], device="cuda")
        outs, lds, strides = [buffer[:, :, k].transpose(0, 1) for k in range(3)], [3 * dim] * 3, [3 * dim * tokens] * 3
    mrr.check(forward(inputs, weights, table, None, None, outs, heads, dim, rot, False, t, "f32", lds=lds, strides=strides))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    dws = [[torch.empty(dim, device="cuda") for _ in range(2)] for _ in range(2)]
    mrr.check(backward(want, total, weights, table, None, dsum, dws[0], heads, dim, rot, False, t, "f32"))
    got = torch.empty_like(dsum)
    mrr.check(backward(outs, total, weights, table, None, got, dws[1], heads, dim, rot, False, t, "f32", lds=lds,
                       strides=strides))
    assert torch.equal(got, dsum) and all(torch.equal(a, b) for a, b in zip(*dws))


def test_weights_and_momentum_as_columns_of_one_buffer():
    announce("muon columns")
    g = seeded(2)
    batch, rows, cols = 3, 70, 90
    grads = [gradient(g, batch, rows, cols) for _ in range(2)]
    w, m = torch.randn(batch, rows, cols, generator=g, device="cuda"), gradient(g, batch, rows, cols)
    m_want, w_want = torch.empty_like(m), [torch.empty_like(w) for _ in range(2)]
    mrr.check(muon(grads, 0.5, m, m_want, 0.9, True, w, w_want, 0.02, 0.1, rows, cols, batch, "f32", "f32"))
    buffer = torch.full((batch, rows, 5, cols), 7.0, device="cuda")
    part = [buffer[:, :, k] for k in range(5)]
    part[0].copy_(w)
    part[1].copy_(m)
    mrr.check(muon(grads, 0.5, part[1], part[2], 0.9, True, part[0], [part[3], part[4]], 0.02, 0.1, rows, cols, batch, "f32", "f32",
                   ld_weight=5 * cols, sw=rows * 5 * cols))
    torch.cuda.synchronize()
    assert torch.equal(part[0], w) and torch.equal(part[1], m) and torch.equal(part[2], m_want)
    # (the norm's sum is taken in another order: its last bit of 64 may differ, and a rounding of X with it)
    for got, want in zip(part[3:], w_want):
        assert float((got - want).abs().max()) <= 2.0 ** -22 * float(want.abs().max())
