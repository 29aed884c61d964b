"""CPU checks of the layer norm entry points: every refusal the header names,
before anything touches a GPU.  Pointers are fake device addresses that no
call here reaches."""
import pytest

import allreduce_reduction_nranks_amd as mrr

BASE = 0x7F0000000000
R, C = 16, 256


def fake(i, off=0):
    return BASE + (i << 24) + off


def fwd(inputs=None, nranks=2, residual=None, weight=None, bias=None, sum=None, out=fake(40), mean=None, rstd=None,
        rows=R, cols=C, ld_in=C, ld_out=C, eps=1e-5, t="bf16", tw="auto"):
    return mrr.mrr_layernorm_fwd([fake(i) for i in range(max(nranks, 1))] if inputs is None else inputs, nranks, residual,
                                 weight, bias, sum, out, mean, rstd, rows, cols, ld_in, ld_out, eps, t, tw, stream=0)


def bwd(dout=fake(0), sum=fake(1), weight=fake(2), mean=fake(3), rstd=fake(4), dres=None, dsum=fake(5), dw=fake(6),
        db=fake(7), rows=R, cols=C, ld_in=C, ld_out=C, t="bf16", tw="auto", ws=fake(8), wsb=None):
    if wsb is None:
        wsb = mrr.mrr_layernorm_bwd_workspace_bytes(rows, cols)
    return mrr.mrr_layernorm_bwd(dout, sum, weight, mean, rstd, dres, dsum, dw, db, rows, cols, ld_in, ld_out, t, tw, ws,
                                 wsb, stream=0)


def test_nothing_to_do_launches_nothing():
    assert fwd(rows=0) == mrr.MRR_OK
    assert bwd(rows=0, dw=None, db=None) == mrr.MRR_OK


@pytest.mark.parametrize("kw,status", [
    (dict(nranks=0), "MRR_EUNSUPPORTED"), (dict(nranks=33), "MRR_EUNSUPPORTED"),
    (dict(t="fp8"), "MRR_EUNSUPPORTED"), (dict(t="bf16", tw="f16"), "MRR_EUNSUPPORTED"),
    (dict(t="f32", tw="bf16"), "MRR_EUNSUPPORTED"), (dict(t="auto"), "MRR_EUNSUPPORTED"),
    (dict(cols=0), "MRR_EINVAL"), (dict(cols=(1 << 20) + 1, ld_in=1 << 21, ld_out=1 << 21), "MRR_EINVAL"),
    (dict(ld_in=C - 1), "MRR_EINVAL"), (dict(ld_out=C - 1), "MRR_EINVAL"), (dict(ld_in=(1 << 31) + 1), "MRR_EINVAL"),
    (dict(rows=(1 << 31) + 1), "MRR_EINVAL"), (dict(eps=-1.0), "MRR_EINVAL"), (dict(eps=float("nan")), "MRR_EINVAL"),
    (dict(out=None), "MRR_EINVAL"), (dict(inputs=[fake(0), 0]), "MRR_EINVAL"),
    (dict(inputs=[fake(0), fake(1, 1)]), "MRR_EALIGN"), (dict(out=fake(40, 1)), "MRR_EALIGN"),
    (dict(residual=fake(9, 1)), "MRR_EALIGN"), (dict(weight=fake(9, 2), tw="f32"), "MRR_EALIGN"),
    (dict(mean=fake(9, 2)), "MRR_EALIGN"),
    (dict(out=fake(0, 2)), "MRR_EOVERLAP"), (dict(out=fake(0), ld_out=C + 1), "MRR_EOVERLAP"),
    (dict(sum=fake(40)), "MRR_EOVERLAP"), (dict(sum=fake(40, C * 2)), "MRR_EOVERLAP"),
    (dict(weight=fake(40)), "MRR_EOVERLAP"), (dict(mean=fake(0)), "MRR_EOVERLAP"),
    (dict(mean=fake(9), rstd=fake(9, 4 * R - 4)), "MRR_EOVERLAP"),
    # columns of one wider buffer: the second half starts inside the first
    (dict(inputs=[fake(0), fake(1)], out=fake(0, 2 * C - 2), ld_in=2 * C, ld_out=2 * C), "MRR_EOVERLAP"),
])
def test_forward_refusals(kw, status):
    assert mrr.STATUS_NAMES[fwd(**kw)] == status


@pytest.mark.parametrize("kw,status", [
    (dict(t="fp8fn"), "MRR_EUNSUPPORTED"), (dict(t="f16", tw="bf16"), "MRR_EUNSUPPORTED"),
    (dict(cols=0), "MRR_EINVAL"), (dict(ld_in=1), "MRR_EINVAL"), (dict(rows=(1 << 31) + 1), "MRR_EINVAL"),
    (dict(dsum=None, dw=None, db=None), "MRR_EINVAL"), (dict(dout=None), "MRR_EINVAL"), (dict(sum=None), "MRR_EINVAL"),
    (dict(mean=None), "MRR_EINVAL"), (dict(rstd=None), "MRR_EINVAL"), (dict(ws=None), "MRR_EINVAL"),
    (dict(wsb=8), "MRR_ESCRATCH"), (dict(ws=fake(8, 8)), "MRR_EALIGN"), (dict(dsum=fake(5, 1)), "MRR_EALIGN"),
    (dict(dw=fake(6, 2), tw="f32"), "MRR_EALIGN"), (dict(rstd=fake(4, 1)), "MRR_EALIGN"),
    (dict(dsum=fake(0, 2)), "MRR_EOVERLAP"), (dict(dsum=fake(0), ld_out=C + 8), "MRR_EOVERLAP"),
    (dict(dw=fake(7)), "MRR_EOVERLAP"), (dict(dw=fake(2)), "MRR_EOVERLAP"), (dict(ws=fake(0)), "MRR_EOVERLAP"),
    (dict(ws=fake(6)), "MRR_EOVERLAP"), (dict(dsum=fake(3)), "MRR_EOVERLAP"),
])
def test_backward_refusals(kw, status):
    assert mrr.STATUS_NAMES[bwd(**kw)] == status


def test_lists_and_tensors_that_are_too_small_are_refused():
    import torch
    with pytest.raises(ValueError):
        fwd(inputs=[fake(0)], nranks=2)
    small, big = torch.empty(R * C - 1, dtype=torch.bfloat16), torch.empty(R * C, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fwd(out=small)
    with pytest.raises(ValueError):
        fwd(inputs=[big, small])
    with pytest.raises(ValueError):
        bwd(dsum=small)
    # a view of a wider tensor spans what its strides say (refused later: not a device pointer's business)
    view = torch.empty(R, 2 * C, dtype=torch.bfloat16)[:, :C]
    assert fwd(inputs=[view, view], ld_in=2 * C, out=None) == mrr.MRR_EINVAL


def test_workspace_size():
    assert mrr.mrr_layernorm_bwd_workspace_bytes(0, 100) == 0
    assert mrr.mrr_layernorm_bwd_workspace_bytes(10, 0) == 0
    one = mrr.mrr_layernorm_bwd_workspace_bytes(1, 4096)
    assert one >= 2 * 4096 * 4
    assert mrr.mrr_layernorm_bwd_workspace_bytes(1 << 30, 4096) <= 1024 * 2 * 4096 * 4


def test_tensors_whose_elements_lie_apart_are_refused():
    import torch
    apart = torch.empty(2 * C, dtype=torch.bfloat16)[::2]
    turned = torch.empty(C, R, dtype=torch.bfloat16).t()
    for kw in (dict(weight=apart), dict(bias=apart), dict(mean=torch.empty(2 * R)[::2]), dict(out=turned),
               dict(inputs=[turned, fake(1)]), dict(inputs=[turned, turned])):
        with pytest.raises(ValueError):
            fwd(**kw)
    for kw in (dict(rstd=torch.empty(2 * R)[::2]), dict(dout=turned), dict(dsum=turned)):
        with pytest.raises(ValueError):
            bwd(**kw)
