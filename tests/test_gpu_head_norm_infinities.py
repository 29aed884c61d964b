"""GPU checks of gradients that are not finite (16-bit training with a scaled loss meets them): where heads do not fill a wave, the
lanes without a head must add nothing to the weights' gradients, not the 0 * inf of the head whose elements they hold."""
import pytest
import torch

import allreduce_reduction_nranks_amd as mrr
from gpu_common import announce
from test_gpu_qknorm import TYPES, backward, randn, seeded, table_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("heads", [(5, 3, 1), (1, 1, 0), (9, 2, 2)])
@pytest.mark.parametrize("dim", [64, 128, 80, 7])
@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
def test_an_infinity_in_the_last_head_stays_one(t, heads, dim, value):
    announce("qk infinite gradient", t, heads, dim, value)
    g = seeded(dim)
    tokens, heads = 9, list(heads)
    h = randn(g, tokens, sum(heads) * dim, t=t).abs() + 1.0
    douts = [randn(g, tokens, n, dim, t=t) for n in heads]
    for d in douts[:2]:
        d[4, -1, 3] = value
    dsum, dws = torch.empty_like(h), [torch.empty(dim, device="cuda") for _ in range(2)]
    mrr.check(backward(douts, h, [None, None], table_of(0), None, dsum, dws, heads, dim, 0, False, t, "f32"))
    other = torch.arange(dim, device="cuda") != 3
    for dw in dws:
        assert float(dw[3]) == value and bool(dw[other].isfinite().all())
