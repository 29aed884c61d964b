"""CPU checks of the head norm entry points: every refusal the header names, before anything
touches a GPU.  Pointers are fake device addresses that no call here reaches."""
import pytest
import torch

import allreduce_reduction_nranks_amd as mrr

BASE = 0x7F0000000000
T, H, D, R = 16, [4, 2, 2], 64, 32
W = sum(H) * D


def fake(i, off=0):
    return BASE + (i << 28) + off


def fwd(inputs=None, nranks=2, qw=fake(50), kw=fake(51), table=fake(52), table_rows=100, positions=fake(53), sum=None,
        outs=(fake(60), fake(61), fake(62)), tokens=T, heads=H, dim=D, rot=R, pairs=False, ld_in=W, lds=(4 * D, 2 * D, 2 * D),
        strides=(D, D, D), eps=1e-6, t="bf16", tw="auto"):
    inputs = [fake(i) for i in range(max(nranks, 1))] if inputs is None else inputs
    return mrr.STATUS_NAMES[mrr.mrr_qknorm_rope_fwd(inputs, nranks, qw, kw, table, table_rows, positions, sum, outs, tokens, heads, dim, rot,
                                                    pairs, ld_in, lds, strides, eps, t, tw, stream=0)]


def bwd(douts=(fake(60), fake(61), fake(62)), sum=fake(0), qw=fake(50), kw=fake(51), table=fake(52), table_rows=100, positions=fake(53),
        dsum=fake(1), dq=fake(70), dk=fake(71), tokens=T, heads=H, dim=D, rot=R, pairs=False, ld_in=W, lds=(4 * D, 2 * D, 2 * D),
        strides=(D, D, D), eps=1e-6, t="bf16", tw="auto", ws=fake(80), wsb=None):
    if wsb is None:
        wsb = mrr.mrr_qknorm_rope_bwd_workspace_bytes(tokens, heads, dim) if heads is not None else 0
    return mrr.STATUS_NAMES[mrr.mrr_qknorm_rope_bwd(douts, sum, qw, kw, table, table_rows, positions, dsum, dq, dk, tokens, heads, dim, rot,
                                                    pairs, ld_in, lds, strides, eps, t, tw, ws, wsb, stream=0)]


SHARED = [
    (dict(t="fp8"), "MRR_EUNSUPPORTED"), (dict(t="auto"), "MRR_EUNSUPPORTED"), (dict(t="bf16", tw="f16"), "MRR_EUNSUPPORTED"),
    (dict(t="f32", tw="bf16"), "MRR_EUNSUPPORTED"),
    (dict(dim=0), "MRR_EINVAL"), (dict(dim=513, ld_in=8 * 513), "MRR_EINVAL"), (dict(rot=31), "MRR_EINVAL"), (dict(rot=66), "MRR_EINVAL"),
    (dict(heads=[0, 0, 0]), "MRR_EINVAL"), (dict(heads=[65536, 1, 1], ld_in=1 << 31), "MRR_EINVAL"), (dict(ld_in=W - 1), "MRR_EINVAL"),
    (dict(ld_in=(1 << 31) + 1), "MRR_EINVAL"), (dict(tokens=(1 << 31) + 1), "MRR_EINVAL"), (dict(eps=-1.0), "MRR_EINVAL"),
    (dict(eps=float("nan")), "MRR_EINVAL"), (dict(table=None), "MRR_EINVAL"), (dict(table_rows=0), "MRR_EINVAL"),
    (dict(positions=None, table_rows=T - 1), "MRR_EINVAL"), (dict(heads=None), "MRR_EINVAL"), (dict(lds=None), "MRR_EINVAL"),
    (dict(strides=None), "MRR_EINVAL"), (dict(strides=(D - 1, D, D)), "MRR_EINVAL"), (dict(lds=(4 * D, 2 * D - 1, 2 * D)), "MRR_EINVAL"),
    (dict(lds=(D, 2 * D, 2 * D), strides=(T * D - 1, D, D)), "MRR_EINVAL"), (dict(lds=(0, 2 * D, 2 * D)), "MRR_EINVAL"),
    (dict(table=fake(52, 2)), "MRR_EALIGN"), (dict(positions=fake(53, 4)), "MRR_EALIGN"), (dict(qw=fake(50, 1)), "MRR_EALIGN"),
    (dict(kw=fake(51, 2), tw="f32"), "MRR_EALIGN"),
]


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(nranks=0), "MRR_EUNSUPPORTED"), (dict(nranks=33), "MRR_EUNSUPPORTED"), (dict(inputs=[fake(0), 0]), "MRR_EINVAL"),
    (dict(outs=(None, None, None)), "MRR_EINVAL"), (dict(outs=None), "MRR_EINVAL"), (dict(inputs=[fake(0), fake(1, 1)]), "MRR_EALIGN"),
    (dict(outs=(fake(60, 1), None, None)), "MRR_EALIGN"), (dict(sum=fake(9, 1)), "MRR_EALIGN"),
    # in another heads' place, in an input's with other strides, or beside it
    (dict(outs=(fake(0, 2), None, None), lds=(W,) * 3), "MRR_EOVERLAP"), (dict(outs=(fake(0), None, None)), "MRR_EOVERLAP"),
    (dict(outs=(None, fake(0), None), lds=(W,) * 3), "MRR_EOVERLAP"), (dict(outs=(fake(60), fake(60), None)), "MRR_EOVERLAP"),
    (dict(outs=(fake(50), None, None)), "MRR_EOVERLAP"), (dict(outs=(fake(52), None, None)), "MRR_EOVERLAP"),
    (dict(outs=(fake(53), None, None)), "MRR_EOVERLAP"), (dict(sum=fake(60)), "MRR_EOVERLAP"), (dict(sum=fake(0, 2 * D)), "MRR_EOVERLAP"),
    (dict(sum=fake(0), outs=(fake(0), None, None), lds=(W,) * 3), "MRR_EOVERLAP"),
    (dict(inputs=[fake(0), fake(0, D * 2)], outs=(fake(0), None, None), lds=(W,) * 3), "MRR_EOVERLAP"),
])
def test_forward_refusals(kw, status):
    assert fwd(**kw) == status


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(sum=None), "MRR_EINVAL"), (dict(dsum=None, dq=None, dk=None), "MRR_EINVAL"), (dict(douts=None), "MRR_EINVAL"),
    (dict(ws=None), "MRR_EINVAL"), (dict(wsb=8), "MRR_ESCRATCH"), (dict(ws=fake(80, 8)), "MRR_EALIGN"), (dict(dsum=fake(1, 1)), "MRR_EALIGN"),
    (dict(dq=fake(70, 2), tw="f32", qw=None, kw=None), "MRR_EALIGN"), (dict(douts=(fake(60, 1), None, None)), "MRR_EALIGN"),
    (dict(dsum=fake(0, 2)), "MRR_EOVERLAP"), (dict(dsum=fake(60)), "MRR_EOVERLAP"), (dict(dq=fake(71)), "MRR_EOVERLAP"),
    (dict(dq=fake(50)), "MRR_EOVERLAP"), (dict(dk=fake(0)), "MRR_EOVERLAP"), (dict(ws=fake(0)), "MRR_EOVERLAP"),
    (dict(ws=fake(70)), "MRR_EOVERLAP"), (dict(dq=fake(52)), "MRR_EOVERLAP"),
])
def test_backward_refusals(kw, status):
    assert bwd(**kw) == status


def test_what_the_header_allows_is_not_refused():
    """(Without a GPU an accepted call ends at its launch.)"""
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real")
    whole = (W,) * 3
    places = [2 * D * k for k in (0, 4, 6)]
    for r in range(2):
        assert fwd(outs=[fake(r, p) for p in places], lds=whole) == "MRR_EHIP"
    assert fwd(sum=fake(1)) == fwd(inputs=[fake(0), fake(0, 2)]) == fwd(rot=0, table=None) == fwd(qw=None, kw=None) == "MRR_EHIP"
    assert fwd(lds=(D, D, 4 * D), strides=(T * D, (T + 3) * D, 2 * D)) == fwd(outs=(None, None, fake(62))) == "MRR_EHIP"
    # columns of one wider buffer
    assert fwd(outs=[fake(60, p) for p in places], lds=whole) == fwd(positions=None) == fwd(heads=[4, 4, 0], lds=(4 * D, 4 * D, 0)) == "MRR_EHIP"
    assert bwd(dsum=fake(0)) == bwd(douts=(None,) * 3) == bwd(dq=None, dk=None, ws=None, wsb=0) == bwd(dsum=None) == "MRR_EHIP"
    assert bwd(tokens=0, sum=None) == "MRR_EHIP"


def test_nothing_to_do_launches_nothing():
    assert fwd(tokens=0) == "MRR_OK"
    assert bwd(tokens=0, dq=None, dk=None) == "MRR_OK"


def test_lists_and_tensors_that_are_too_small_are_refused():
    big, small = torch.empty(T, W, dtype=torch.bfloat16), torch.empty(T * W - 1, dtype=torch.bfloat16)
    out = torch.empty(T, 4, D, dtype=torch.bfloat16)
    for kw in (dict(inputs=[fake(0)]), dict(inputs=[big, small]), dict(outs=(fake(0), fake(1))), dict(heads=[4, 2]), dict(lds=(1, 2)),
               dict(outs=(out[:-1], None, None)), dict(outs=(out, None, None), lds=(5 * D, 1, 1)), dict(outs=(out.transpose(1, 2), None, None)),
               dict(qw=torch.empty(D - 1, dtype=torch.bfloat16)), dict(table=torch.empty(99, R)), dict(positions=torch.zeros(T - 1, dtype=torch.int64)),
               dict(sum=small)):
        with pytest.raises(ValueError):
            fwd(**kw)
    for kw in (dict(dsum=small), dict(sum=small), dict(douts=(out[1:], None, None)), dict(dq=torch.empty(D - 1, dtype=torch.bfloat16)),
               dict(ws=torch.empty(8, dtype=torch.uint8), wsb=16)):
        with pytest.raises(ValueError):
            bwd(**kw)


def test_workspace_size():
    assert mrr.mrr_qknorm_rope_bwd_workspace_bytes(10, H, 0) == mrr.mrr_qknorm_rope_bwd_workspace_bytes(10, H, 513) == 0
    assert 2 * 128 * 4 <= mrr.mrr_qknorm_rope_bwd_workspace_bytes(1 << 30, H, 128) <= 1 << 21
