"""CPU checks of the cross entropy workspaces: no room for weights that a call reads where they
are, and a refusal where a call has to lay them out after all.  Pointers are fake device
addresses that no call here reaches."""
import pytest

import allreduce_reduction_nranks_amd as mrr

BASE = 0x7F0000000000
MiB = 1 << 20


def fake(i, off=0):
    return BASE + (i << 36) + off


def sizes(tokens, cols, rows, t, backward):
    return (mrr.mrr_linear_xent_workspace_bytes(tokens, cols, rows, len(rows), t, backward),
            mrr.mrr_linear_xent_workspace_bytes_in_place(tokens, cols, rows, len(rows), t, backward))


def call(backward, wsb, tokens=40, cols=128, rows=(700, 300), t="bf16", hidden=fake(0), weights=(fake(1), fake(2)), ldh=None,
         ldw=None):
    ldh, ldw, rows = ldh or cols, ldw or cols, list(rows)
    if backward:
        st = mrr.mrr_linear_xent_bwd(hidden, list(weights), rows, 2, fake(3), -100, fake(5), fake(7), 1, fake(8),
                                     [fake(9), fake(10)], tokens, cols, ldh, ldw, t, fake(6), wsb, stream=0)
    else:
        st = mrr.mrr_linear_xent_fwd(hidden, list(weights), rows, 2, fake(3), -100, fake(4), fake(5), tokens, cols, ldh, ldw, t,
                                     fake(6), wsb, stream=0)
    return mrr.STATUS_NAMES[st]


@pytest.mark.parametrize("tokens,cols,vocab,t", [(1, 4096, 32000, "bf16"), (1, 4096, 128256, "bf16"), (4, 1023, 50257, "f16"),
                                                 (1, 4096, 32000, "f32"), (130, 520, 3003, "f32")])
def test_a_forward_of_few_tokens_has_no_room_for_weights(tokens, cols, vocab, t):
    # pairs of 8 bytes for every 16 rows and token, and what is rounded up
    bound = (vocab / 16 + 64) * 8 * tokens + 4096
    assert max(sizes(tokens, cols, [vocab // 2, vocab - vocab // 2], t, False)) <= bound


@pytest.mark.parametrize("tokens,cols,vocab", [(16, 4096, 128256), (64, 1024, 32000), (700, 1600, 50240), (4096, 4096, 128256)])
def test_calls_in_place_have_no_room_for_weights(tokens, cols, vocab):
    rows = [vocab // 8] * 8
    for backward in (False, True):
        every, in_place = sizes(tokens, cols, rows, "bf16", backward)
        laid = 2 * cols * min(vocab, (64 * MiB) // cols)  # at least: a quarter of a piece, or all
        assert in_place + laid <= every
    # pairs for every 64 rows (of up to 64 tokens 16) and token
    assert sizes(tokens, cols, rows, "bf16", False)[1] <= (vocab / (16 if tokens <= 64 else 64) + 64 * 8) * 8 * tokens + 8 * tokens + 4096


@pytest.mark.parametrize("tokens,cols,t", [(700, 1023, "f16"), (2000, 128, "f32"), (300, 33, "bf16")])
def test_sizes_that_are_never_in_place_have_one_number(tokens, cols, t):
    for backward in (False, True):
        every, in_place = sizes(tokens, cols, [30000, 1], t, backward)
        assert every == in_place


def test_no_size_for_what_is_refused():
    for f in (mrr.mrr_linear_xent_workspace_bytes_in_place, mrr.mrr_linear_xent_workspace_bytes):
        assert f(0, 64, [5], 1, "bf16", False) == f(4, 0, [5], 1, "bf16", False) == f(4, 64, [0], 1, "bf16", True) == 0
        assert f(4, 64, [5], 1, "fp8", True) == f(4, 64, [5], 0, "bf16", True) == 0


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("tokens", [40, 300])
def test_the_smaller_workspace_is_for_operands_in_place(tokens, backward):
    """(Without a GPU an accepted call ends at its launch.)"""
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real")
    every, in_place = sizes(tokens, 128, [700, 300], "bf16", backward)
    assert in_place < every
    assert call(backward, in_place, tokens) == "MRR_EHIP"
    assert call(backward, in_place - 1, tokens) == "MRR_ESCRATCH"
    for kw in (dict(weights=(fake(1), fake(2, 8))), dict(ldw=129), dict(ldw=(1 << 22) + 8)):
        assert call(backward, every - 1, tokens, **kw) == "MRR_ESCRATCH"
        assert call(backward, every, tokens, **kw) == "MRR_EHIP"
    # a backward gathers the hidden states in any case
    for kw in (dict(hidden=fake(0, 2)), dict(ldh=129)):
        assert call(backward, in_place, tokens, **kw) == ("MRR_EHIP" if backward else "MRR_ESCRATCH")
