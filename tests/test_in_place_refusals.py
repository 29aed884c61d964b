"""CPU checks of which output may take which input's place in the norm and cross entropy calls:
each output has its own list, also where one row makes a vector and a matrix look alike.
Pointers are fake device addresses that no call here reaches."""
import pytest

import allreduce_reduction_nranks_amd as mrr

BASE = 0x7F0000000000


def fake(i, off=0):
    return BASE + (i << 32) + off


def norm_fwd(rows, cols, inputs=(fake(0), fake(1)), residual=fake(2), sum=None, out=fake(3), mean=None, rstd=None):
    return mrr.STATUS_NAMES[mrr.mrr_layernorm_fwd(list(inputs), len(inputs), residual, None, None, sum, out, mean, rstd, rows,
                                                  cols, cols, cols, 1e-5, "f32", "f32", stream=0)]


def norm_bwd(t, rows=1, cols=64, dres=fake(2), dsum=fake(5), dw=fake(6), db=fake(7), ws=fake(8)):
    n = mrr.mrr_layernorm_bwd_workspace_bytes(rows, cols)
    return mrr.STATUS_NAMES[mrr.mrr_layernorm_bwd(fake(0), fake(1), None, fake(3), fake(4), dres, dsum, dw, db, rows, cols, cols,
                                                  cols, t, "auto", ws, n, stream=0)]


def xent_bwd(t, rows, tokens, dh=fake(8), dw=(fake(9), fake(10)), cols=64):
    n = mrr.mrr_linear_xent_workspace_bytes(tokens, cols, rows, 2, t, True)
    return mrr.STATUS_NAMES[mrr.mrr_linear_xent_bwd(fake(0), [fake(1), fake(2)], rows, 2, fake(3), -100, fake(5), fake(7), 1, dh,
                                                    list(dw), tokens, cols, cols, cols, t, fake(6), n, stream=0)]


@pytest.mark.parametrize("which", [0, 1, 2])
@pytest.mark.parametrize("name", ["mean", "rstd"])
def test_the_statistics_of_a_norm_take_no_input_s_place(name, which):
    # one row of one f32 element: input, residual and statistics are 4 bytes each
    assert norm_fwd(1, 1, **{name: fake(which)}) == "MRR_EOVERLAP"


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("which", [0, 1, 2])
@pytest.mark.parametrize("name", ["dw", "db"])
def test_a_weight_gradient_takes_no_input_s_place(name, which, t):
    assert norm_bwd(t, **{name: fake(which)}) == "MRR_EOVERLAP"


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("tokens", [1, 40, 300])
@pytest.mark.parametrize("shard", [0, 1])
def test_a_shard_s_gradient_does_not_take_the_hidden_states_place(tokens, shard, t):
    rows, dw = [7, 7], [fake(9), fake(10)]
    rows[shard], dw[shard] = tokens, fake(0)
    assert xent_bwd(t, rows, tokens, dw=dw) == "MRR_EOVERLAP"


def test_what_the_header_allows_is_not_refused():
    """(Without a GPU an accepted call ends at its launch.)"""
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real")
    for which in (0, 1, 2):
        assert norm_fwd(1, 1, sum=fake(which)) == norm_fwd(1, 1, out=fake(which)) == "MRR_EHIP"
        assert norm_bwd("bf16", dsum=fake(which)) == norm_bwd("bf16", rows=5, dsum=fake(which)) == "MRR_EHIP"
    assert norm_fwd(3, 8, sum=fake(0), out=fake(1)) == "MRR_EHIP"
    assert xent_bwd("bf16", [7, 7], 7, dh=fake(0)) == "MRR_EHIP"
