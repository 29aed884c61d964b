"""CPU checks of the loss gradients' stride: what a tensor's own strides hold has to cover what
the call's stride reaches, however many elements the tensor counts."""
import pytest
import torch

import allreduce_reduction_nranks_amd as mrr

T, C, ROWS = 4096, 64, [100, 28]
BASE = 0x7F0000000000


def fake(i):
    return BASE + (i << 32)


def bwd(dloss, stride, tokens=T):
    n = mrr.mrr_linear_xent_workspace_bytes(tokens, C, ROWS, 2, "bf16", True)
    # no output: refused by the C entry point once the arguments have passed
    return mrr.mrr_linear_xent_bwd(fake(0), [fake(1), fake(2)], ROWS, 2, fake(3), -100, fake(4), dloss, stride, None, None, tokens,
                                   C, C, C, "bf16", fake(5), n, stream=0)


@pytest.mark.parametrize("dloss,stride", [
    (torch.ones(1).expand(T), 1), (torch.ones(()).expand(T), 1), (torch.ones(2).repeat_interleave(1)[:1].expand(T), 2),
    (torch.ones(T, 1).expand(T, 3), 3), (torch.ones(1, 5).expand(T, 5), 5), (torch.ones(T)[::2], 1), (torch.ones(T), 2),
    (torch.ones(0), 0),
])
def test_a_gradient_that_ends_before_the_last_token_is_refused(dloss, stride):
    with pytest.raises(ValueError):
        bwd(dloss, stride)


@pytest.mark.parametrize("dloss,stride", [
    (torch.ones(1).expand(T), 0), (torch.ones(()), 0), (torch.ones(T), 1), (torch.ones(T, 5), 5), (torch.ones(T, 5)[:, 2], 5),
    (torch.ones(2 * T)[::2], 2), (fake(6), 7),
])
def test_a_gradient_that_holds_every_token_s_is_taken(dloss, stride):
    assert bwd(dloss, stride) == mrr.MRR_EINVAL


def test_no_tokens_need_no_gradient():
    assert bwd(torch.ones(0), 1, tokens=0) == mrr.MRR_EINVAL
