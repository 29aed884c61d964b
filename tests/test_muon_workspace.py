"""CPU checks of the update's workspace for the defaults of mrr_muon_step: weights of the gradients' type."""
import pytest
import torch

import allreduce_reduction_nranks_amd as mrr

BASE = 0x7F0000000000


@pytest.mark.parametrize("products", ["auto", "f32", "f16"])
@pytest.mark.parametrize("rows,cols,batch", [(96, 160, 2), (700, 300, 1), (40, 900, 3), (1, 1, 1)])
def test_the_default_weight_type_has_a_size(rows, cols, batch, products):
    for nesterov in (True, False):
        n = mrr.mrr_muon_workspace_bytes(rows, cols, batch, "auto", products, nesterov)
        assert n and all(n == mrr.mrr_muon_workspace_bytes(rows, cols, batch, t, products, nesterov) for t in ("bf16", "f16", "f32"))


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
def test_the_size_serves_the_call(t):
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real")
    a = [BASE + (k << 34) for k in range(6)]

    def step(n):
        return mrr.STATUS_NAMES[mrr.mrr_muon_step([a[0]], 1, 1.0, None, a[1], 0.9, True, a[2], [a[3]], 0.02, 0.0, 96, 160, 160, 160, 2, 15360,
                                                  15360, 5, None, 1e-7, t, workspace=a[4], workspace_bytes=n, stream=0)]
    n = mrr.mrr_muon_workspace_bytes(96, 160, 2, "auto")
    assert step(n) == "MRR_EHIP" and step(n - 1) == "MRR_ESCRATCH"


def test_types_without_an_update_have_none():
    assert mrr.mrr_muon_workspace_bytes(96, 160, 2, "fp8") == mrr.mrr_orthogonalize_workspace_bytes(96, 160, 2, "auto") == 0
