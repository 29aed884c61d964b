"""CPU checks of the cross entropy entry points: every refusal the header names,
before anything touches a GPU.  Pointers are fake device addresses that no call
here reaches."""
import pytest

import allreduce_reduction_nranks_amd as mrr

BASE = 0x7F0000000000
T, C, ROWS = 16, 64, [100, 28]


def fake(i, off=0):
    return BASE + (i << 32) + off


def bytes_of(tokens, cols, rows, n, t, backward):
    return mrr.mrr_linear_xent_workspace_bytes(tokens, cols, rows, n, t, backward)


def fwd(hidden=fake(0), weights=(fake(1), fake(2)), rows=ROWS, n=2, targets=fake(3), loss=fake(4), lse=fake(5), tokens=T,
        cols=C, ldh=C, ldw=C, t="bf16", ws=fake(6), wsb=None):
    if wsb is None:
        wsb = bytes_of(tokens, cols, rows, n, t, False)
    return mrr.mrr_linear_xent_fwd(hidden, weights, rows, n, targets, -100, loss, lse, tokens, cols, ldh, ldw, t, ws, wsb,
                                   stream=0)


def bwd(hidden=fake(0), weights=(fake(1), fake(2)), rows=ROWS, n=2, targets=fake(3), lse=fake(5), dloss=fake(7), stride=1,
        dh=fake(8), dw=[fake(9 + i) for i in range(33)], tokens=T, cols=C, ldh=C, ldw=C, t="bf16", ws=fake(6), wsb=None):
    if wsb is None:
        wsb = bytes_of(tokens, cols, rows, n, t, True)
    return mrr.mrr_linear_xent_bwd(hidden, weights, rows, n, targets, -100, lse, dloss, stride, dh, dw, tokens, cols, ldh,
                                   ldw, t, ws, wsb, stream=0)


SHARED = [
    (dict(n=0), "MRR_EUNSUPPORTED"), (dict(n=33, rows=[1] * 33, weights=[fake(1)] * 33), "MRR_EUNSUPPORTED"),
    (dict(t="fp8"), "MRR_EUNSUPPORTED"), (dict(t="auto"), "MRR_EUNSUPPORTED"),
    (dict(cols=0), "MRR_EINVAL"), (dict(cols=(1 << 20) + 1, ldh=1 << 21, ldw=1 << 21), "MRR_EINVAL"),
    (dict(tokens=(1 << 24) + 1), "MRR_EINVAL"), (dict(rows=[0, 0]), "MRR_EINVAL"), (dict(rows=[1 << 30, 1]), "MRR_EINVAL"),
    (dict(rows=[(1 << 63), 1 << 63]), "MRR_EINVAL"), (dict(ldh=C - 1), "MRR_EINVAL"), (dict(ldw=C - 1), "MRR_EINVAL"),
    (dict(ldw=(1 << 31) + 1), "MRR_EINVAL"), (dict(hidden=None), "MRR_EINVAL"), (dict(weights=None), "MRR_EINVAL"),
    (dict(weights=[fake(1), 0]), "MRR_EINVAL"), (dict(targets=None), "MRR_EINVAL"), (dict(ws=None), "MRR_EINVAL"),
    (dict(wsb=0), "MRR_ESCRATCH"), (dict(ws=fake(6, 8)), "MRR_EALIGN"), (dict(hidden=fake(0, 1)), "MRR_EALIGN"),
    (dict(targets=fake(3, 4)), "MRR_EALIGN"), (dict(weights=[fake(1), fake(2, 1)]), "MRR_EALIGN"),
    (dict(t="f32", weights=[fake(1, 2), fake(2)]), "MRR_EALIGN"), (dict(ws=fake(0)), "MRR_EOVERLAP"),
    (dict(ws=fake(1)), "MRR_EOVERLAP"), (dict(ws=fake(3)), "MRR_EOVERLAP"),
]


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(loss=None, lse=None), "MRR_EINVAL"), (dict(loss=fake(4, 2)), "MRR_EALIGN"), (dict(lse=fake(5, 1)), "MRR_EALIGN"),
    (dict(loss=fake(5, 4 * T - 4)), "MRR_EOVERLAP"), (dict(lse=fake(0)), "MRR_EOVERLAP"), (dict(loss=fake(3)), "MRR_EOVERLAP"),
    (dict(loss=fake(6)), "MRR_EOVERLAP"),
])
def test_forward_refusals(kw, status):
    assert mrr.STATUS_NAMES[fwd(**kw)] == status


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(dh=None, dw=None), "MRR_EINVAL"), (dict(dh=None, dw=[None, None]), "MRR_EINVAL"), (dict(lse=None), "MRR_EINVAL"),
    (dict(dloss=None), "MRR_EINVAL"), (dict(stride=(1 << 31) + 1), "MRR_EINVAL"), (dict(dloss=fake(7, 2)), "MRR_EALIGN"),
    (dict(dh=fake(8, 1)), "MRR_EALIGN"), (dict(dw=[fake(9, 1), fake(10)]), "MRR_EALIGN"),
    (dict(dh=fake(0, 2)), "MRR_EOVERLAP"), (dict(dh=fake(1)), "MRR_EOVERLAP"), (dict(dw=[fake(1), fake(10)]), "MRR_EOVERLAP"),
    (dict(dw=[fake(9), fake(9)]), "MRR_EOVERLAP"), (dict(dw=[fake(0), fake(10)]), "MRR_EOVERLAP"),
    (dict(dh=fake(6)), "MRR_EOVERLAP"), (dict(dw=[fake(5), fake(10)]), "MRR_EOVERLAP"),
    (dict(dloss=fake(8, T * C * 2 - 4)), "MRR_EOVERLAP"),
])
def test_backward_refusals(kw, status):
    assert mrr.STATUS_NAMES[bwd(**kw)] == status


def test_nothing_to_do_launches_nothing():
    assert fwd(tokens=0, hidden=None, targets=None, ws=None) == mrr.MRR_OK
    assert bwd(tokens=0, hidden=None, targets=None, ws=None, dw=None) == mrr.MRR_OK


def test_lists_and_tensors_that_are_too_small_are_refused():
    import torch
    small = torch.empty(T * C - 1, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fwd(rows=[100])
    with pytest.raises(ValueError):
        fwd(weights=[fake(1)])
    with pytest.raises(ValueError):
        fwd(hidden=small)
    with pytest.raises(ValueError):
        fwd(weights=[fake(1), small])
    with pytest.raises(ValueError):
        fwd(loss=torch.empty(T - 1))
    with pytest.raises(ValueError):
        fwd(targets=torch.empty(T, dtype=torch.int32))
    with pytest.raises(ValueError):
        bwd(dh=small)
    with pytest.raises(ValueError):
        bwd(dw=[small, fake(10)])
    with pytest.raises(ValueError):
        bwd(dloss=torch.empty(T), stride=2)
    with pytest.raises(ValueError):
        bwd(ws=torch.empty(8, dtype=torch.uint8), wsb=1 << 20)


def test_workspace_size():
    assert bytes_of(0, C, ROWS, 2, "bf16", False) == 0
    assert bytes_of(4, 0, ROWS, 2, "bf16", False) == 0
    assert bytes_of(4, C, [0, 0], 2, "bf16", True) == 0
    # the logits of this call would take 2 GiB in 32 bits: neither direction keeps them
    big = [bytes_of(4096, 4096, [16032] * 8, 8, "bf16", b) for b in (False, True)]
    assert 0 < big[0] < big[1] < (3 << 29)


def test_tensors_whose_elements_lie_apart_are_refused():
    import torch
    turned = torch.empty(C, T, dtype=torch.bfloat16).t()
    wide = torch.empty(C, 200, dtype=torch.bfloat16).t()
    for kw in (dict(hidden=turned), dict(weights=[wide, fake(2)]), dict(loss=torch.empty(2 * T)[::2]),
               dict(targets=torch.empty(2 * T, dtype=torch.int64)[::2])):
        with pytest.raises(ValueError):
            fwd(**kw)
    for kw in (dict(dh=turned), dict(dw=[wide, fake(10)]), dict(lse=torch.empty(2 * T)[::2])):
        with pytest.raises(ValueError):
            bwd(**kw)
