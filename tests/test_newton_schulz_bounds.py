"""Coefficients at the limits that the f16 parts of mrr_orthogonalize set, and past them, on the CPU."""
import pytest
import torch

import allreduce_reduction_nranks_amd as mrr

BASE = 0x7F0000000000


def orth(co, steps):
    n = mrr.mrr_orthogonalize_workspace_bytes(96, 160, 1, "bf16")
    return mrr.STATUS_NAMES[mrr.mrr_orthogonalize(BASE, BASE + (1 << 34), 96, 160, 160, 160, 1, 0, 0, steps, co, 1e-7, "bf16", "auto",
                                                  BASE + (2 << 34), n, stream=0)]


@pytest.mark.parametrize("co,steps,refused", [
    ((7.49, 0.0, 0.0), 1, False),                       # nothing follows
    ((7.40, 0.0, 0.0, 1.0, 0.0, 0.0), 2, False),        # 7.474 with 1 % for roundings
    ((7.43, 0.0, 0.0, 1.0, 0.0, 0.0), 2, True),         # 7.504
    ((2.7, 0.0, 0.0, 2.7, 0.0, 0.0, 1.0, 0.0, 0.0), 3, False),   # 2.7 2.7 1.01^2 = 7.436
    ((2.72, 0.0, 0.0, 2.72, 0.0, 0.0, 1.0, 0.0, 0.0), 3, True),  # 7.547
    # b x + c x^2 at x = 1.01^2: just under and over 1000; the value after, 1 + b, is not used
    ((1.0, 0.0, 0.0, 1.0, 980.0, 0.0), 2, False),       # 999.7
    ((1.0, 0.0, 0.0, 1.0, 981.0, 0.0), 2, True),        # 1000.7
])
def test_limits(co, steps, refused):
    if torch.cuda.is_available() and not refused:
        pytest.skip("the addresses are not real")
    assert orth(co, steps) == ("MRR_EINVAL" if refused else "MRR_EHIP")
