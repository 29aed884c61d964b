"""GPU checks of the heads that f32 squares hold a norm of, and of what becomes of the others: a head's squares sum to at most
2^128 (1 - 2^-25), so that head_dim equal elements go up to 2^64 / sqrt(head_dim) = 1.8e19 / sqrt(head_dim)."""
import pytest
import torch

import allreduce_reduction_nranks_amd as mrr
from gpu_common import announce
from test_gpu_qknorm import TYPES, backward, empty_outs, randn, seeded, table_of

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def normed(h, heads, dim, eps):
    outs = empty_outs(len(h), heads, dim, "f32")
    mrr.check(mrr.mrr_qknorm_rope_fwd([h], 1, None, None, table_of(0), 1, None, None, outs, len(h), heads, dim, 0, False, sum(heads) * dim,
                                      [n * dim for n in heads], [dim] * 3, eps, "f32"))
    return outs


@pytest.mark.parametrize("dim", [4, 64, 128, 172, 512])
def test_large_elements(dim):
    announce("qk large elements", dim)
    heads = [2, 1, 1]
    limit = 2.0 ** 64 / dim ** 0.5
    sign = torch.where(torch.rand(3, 4 * dim, generator=seeded(dim), device="cuda") < 0.5, -1.0, 1.0)
    q, k, v = normed(sign * (limit * 0.99), heads, dim, 1e-6)
    want = sign.view(3, 4, dim)
    for got, w in ((q, want[:, :2]), (k, want[:, 2:3])):
        assert float((got - w).abs().max()) <= 32 * U
    # past it: zeros, and gradients of zero
    h = sign * (limit * 1.01)
    q, k, v = normed(h, heads, dim, 1e-6)
    assert not bool(q.any()) and not bool(k.any()) and torch.equal(v.flatten(1), h[:, 3 * dim:])
    g = seeded(dim + 1)
    douts = [randn(g, 3, n, dim) for n in heads]
    dsum, dws = torch.full_like(h, 7.0), [torch.full((dim,), 7.0, device="cuda") for _ in range(2)]
    mrr.check(backward(douts, h, [None, None], table_of(0), None, dsum, dws, heads, dim, 0, False, "f32", "f32"))
    assert not bool(dsum[:, :3 * dim].any()) and not any(bool(d.any()) for d in dws)


@pytest.mark.parametrize("dim", [4, 128])
def test_small_elements_without_eps(dim):
    announce("qk small elements", dim)
    heads = [2, 1, 1]
    x = randn(seeded(dim), 3, 4 * dim)
    x = torch.where(x < 0, x - 1.0, x + 1.0) * 1e-18  # squares of 1e-36 and more: 27 bits above f32's smallest
    q, k, v = normed(x, heads, dim, 0.0)
    h = x.double().view(3, 4, dim)
    want = h / h.square().mean(-1, keepdim=True).sqrt()
    assert float((q - want[:, :2]).abs().div(want[:, :2].abs()).max()) <= 32 * U
    assert float((k - want[:, 2:3]).abs().div(want[:, 2:3].abs()).max()) <= 32 * U
    q, k, v = normed(torch.zeros_like(x), heads, dim, 0.0)
    assert bool(q.isnan().all()) and bool(k.isnan().all()) and not bool(v.any())
