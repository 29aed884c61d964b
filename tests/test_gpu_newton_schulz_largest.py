"""GPU check of the largest matrix that a call takes, 65536 x 65536: one element in each row and column, whose result is the
polynomial of each element by itself."""
import pytest
import torch

import allreduce_reduction_nranks_amd as mrr
from gpu_common import announce
from test_gpu_muon import CO, orth, seeded

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("products", ["auto", "f16"])
def test_largest(products):
    n = 65536
    announce("orth largest", products)
    if torch.cuda.mem_get_info()[0] < 130 << 30:
        pytest.skip("needs 130 GiB of GPU memory")
    g = seeded(1)
    where = torch.randperm(n, generator=g, device="cuda")
    rows = torch.arange(n, device="cuda")
    v = (torch.randn(n, generator=g, device="cuda") + 3.0).bfloat16()
    x = torch.zeros(n, n, dtype=torch.bfloat16, device="cuda")
    x[rows, where] = v
    mrr.check(orth(x, x, n, n, 1, "bf16", products, CO, 1, 0.0))
    s = v.double() / v.double().norm()
    want = s * (CO[0] + CO[1] * s ** 2 + CO[2] * s ** 4)
    # s is about 2^-8: B X, which products of 11 bits round, is 2^-15 of the result
    assert bool(((x[rows, where].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -18) * want.abs()).all())
    x[rows, where] = 0
    assert not bool(x.any())
