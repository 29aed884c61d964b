"""CPU checks of mrr_orthogonalize and mrr_muon_step: every refusal the header names, before
anything touches a GPU.  Pointers are fake device addresses that no call here reaches."""
import pytest
import torch

import allreduce_reduction_nranks_amd as mrr

BASE = 0x7F0000000000
R, C, B = 96, 160, 2
N = R * C


def fake(i, off=0):
    return BASE + (i << 34) + off


def orth(x=fake(0), out=fake(1), rows=R, cols=C, ld_in=C, ld_out=C, batch=B, sin=N, sout=N, steps=5, co=None, eps=1e-7, t="bf16",
         products="auto", ws=fake(2), wsb=None):
    if wsb is None:
        wsb = mrr.mrr_orthogonalize_workspace_bytes(rows, cols, batch, t, products)
    return mrr.STATUS_NAMES[mrr.mrr_orthogonalize(x, out, rows, cols, ld_in, ld_out, batch, sin, sout, steps, co, eps, t, products, ws, wsb,
                                                  stream=0)]


def muon(grads=(fake(0), fake(1)), nranks=2, scale=0.5, m=fake(2), m_out=fake(3), mu=0.9, nesterov=True, w=fake(4),
         w_out=(fake(5), fake(6)), rate=0.02, decay=0.0, rows=R, cols=C, ld_grad=C, ld_weight=C, batch=B, sg=N, sw=N, steps=5, co=None,
         eps=1e-7, tg="bf16", tw="f32", products="auto", ws=fake(7), wsb=None):
    if wsb is None:
        wsb = mrr.mrr_muon_workspace_bytes(rows, cols, batch, tw if tw != "auto" else tg, products, nesterov)
    return mrr.STATUS_NAMES[mrr.mrr_muon_step(grads, nranks, scale, m, m_out, mu, nesterov, w, w_out, rate, decay, rows, cols, ld_grad,
                                              ld_weight, batch, sg, sw, steps, co, eps, tg, tw, products, ws, wsb, stream=0)]


SHARED = [
    (dict(products="bf16"), "MRR_EUNSUPPORTED"), (dict(products="fp8"), "MRR_EUNSUPPORTED"),
    (dict(rows=0), "MRR_EINVAL"), (dict(cols=0), "MRR_EINVAL"), (dict(rows=65537), "MRR_EINVAL"), (dict(batch=65536), "MRR_EINVAL"),
    (dict(steps=0), "MRR_EINVAL"), (dict(steps=65), "MRR_EINVAL"), (dict(eps=-1e-9), "MRR_EINVAL"), (dict(eps=float("nan")), "MRR_EINVAL"),
    (dict(eps=float("inf")), "MRR_EINVAL"), (dict(ws=None), "MRR_EINVAL"), (dict(wsb=100), "MRR_ESCRATCH"), (dict(ws=fake(7, 8)), "MRR_EALIGN"),
    (dict(co=(8.0, 0.0, 0.0) * 5), "MRR_EINVAL"),       # 8, then 64
    (dict(co=(1.0, 999.0, 1.0) * 5), "MRR_EINVAL"), (dict(co=(float("nan"), 0.0, 0.0) * 5), "MRR_EINVAL"),
    (dict(co=(3.0, float("inf"), 0.0) * 5), "MRR_EINVAL"),
    (dict(co=(2.0, -1.5, 0.5, 1.0, 0.0, 0.0, 9.0, 0.0, 0.0, 1.0, 0.0, 0.0, 1.0, 0.0, 0.0)), "MRR_EINVAL"),
]


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(t="fp8"), "MRR_EUNSUPPORTED"), (dict(t="auto"), "MRR_EUNSUPPORTED"), (dict(x=None), "MRR_EINVAL"), (dict(out=None), "MRR_EINVAL"),
    (dict(ld_in=C - 1), "MRR_EINVAL"), (dict(ld_out=(1 << 31) + 1), "MRR_EINVAL"), (dict(sin=(1 << 40) + 1), "MRR_EINVAL"),
    (dict(x=fake(0, 1)), "MRR_EALIGN"), (dict(out=fake(1, 1)), "MRR_EALIGN"),
    (dict(sout=N - 1), "MRR_EOVERLAP"), (dict(sout=0), "MRR_EOVERLAP"), (dict(ld_out=2 * C - 1, sout=C), "MRR_EOVERLAP"),
    (dict(out=fake(0, 2)), "MRR_EOVERLAP"), (dict(out=fake(0), ld_out=C + 1, sout=2 * N), "MRR_EOVERLAP"), (dict(ws=fake(0)), "MRR_EOVERLAP"),
    (dict(ws=fake(1)), "MRR_EOVERLAP"), (dict(out=fake(0), sin=0), "MRR_EOVERLAP"),
])
def test_orthogonalize_refusals(kw, status):
    assert orth(**kw) == status


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(nranks=0), "MRR_EUNSUPPORTED"), (dict(nranks=33, grads=[fake(0)] * 33, w_out=[fake(5)] * 33), "MRR_EUNSUPPORTED"),
    (dict(tg="fp8"), "MRR_EUNSUPPORTED"), (dict(tw="fp8"), "MRR_EUNSUPPORTED"), (dict(tg="auto", tw="auto"), "MRR_EUNSUPPORTED"),
    (dict(grads=(fake(0), None)), "MRR_EINVAL"), (dict(w_out=(fake(5), None)), "MRR_EINVAL"), (dict(w=None), "MRR_EINVAL"),
    (dict(m_out=None), "MRR_EINVAL"), (dict(scale=float("inf")), "MRR_EINVAL"), (dict(mu=float("nan")), "MRR_EINVAL"),
    (dict(rate=float("nan")), "MRR_EINVAL"), (dict(decay=float("inf")), "MRR_EINVAL"), (dict(ld_grad=C - 1), "MRR_EINVAL"),
    (dict(ld_weight=C - 1), "MRR_EINVAL"), (dict(sw=(1 << 40) + 1), "MRR_EINVAL"),
    (dict(grads=(fake(0, 1), fake(1))), "MRR_EALIGN"), (dict(m=fake(2, 2)), "MRR_EALIGN"), (dict(m_out=fake(3, 2)), "MRR_EALIGN"),
    (dict(w=fake(4, 2)), "MRR_EALIGN"), (dict(w_out=(fake(5), fake(6, 2))), "MRR_EALIGN"),
    (dict(w_out=(fake(5), fake(5))), "MRR_EOVERLAP"), (dict(w_out=(fake(4, 4), fake(6))), "MRR_EOVERLAP"), (dict(sw=N - 1), "MRR_EOVERLAP"),
    (dict(w_out=(fake(0), fake(6))), "MRR_EOVERLAP"), (dict(m_out=fake(2, 4)), "MRR_EOVERLAP"), (dict(m_out=fake(4)), "MRR_EOVERLAP"),
    (dict(m_out=fake(0)), "MRR_EOVERLAP"), (dict(m_out=fake(5)), "MRR_EOVERLAP"), (dict(m_out=fake(7)), "MRR_EOVERLAP"),
    (dict(w_out=(fake(2), fake(6))), "MRR_EOVERLAP"), (dict(w_out=(fake(3), fake(6))), "MRR_EOVERLAP"), (dict(ws=fake(4)), "MRR_EOVERLAP"),
])
def test_muon_refusals(kw, status):
    assert muon(**kw) == status


def test_what_the_header_allows_is_not_refused():
    """(Without a GPU an accepted call ends at its launch.)"""
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real")
    assert orth(out=fake(0)) == orth(sin=0) == orth(sin=7) == orth(batch=1, sout=0) == "MRR_EHIP"
    assert orth(ld_out=2 * C, sout=C) == orth(x=fake(0), out=fake(0), ld_in=2 * C, ld_out=2 * C, sin=C, sout=C) == "MRR_EHIP"
    assert orth(products="f32") == orth(t="f32", products="f16") == orth(co=(1.5, -0.5, 0.0) * 5) == orth(co=(7.0, 0.0, 0.0), steps=1) == "MRR_EHIP"
    assert orth(co=(2.0, -1.5, 0.5) * 2 + (3.4445, -4.7750, 2.0315) * 3) == "MRR_EHIP"
    assert muon(m=None) == muon(m_out=fake(2)) == muon(w_out=(fake(4), fake(6))) == muon(tw="auto") == muon(nesterov=False) == "MRR_EHIP"
    assert muon(grads=(fake(0), fake(0))) == muon(sg=0) == muon(tg="f32", tw="bf16") == "MRR_EHIP"


def test_nothing_to_do_launches_nothing():
    assert orth(batch=0) == muon(batch=0) == "MRR_OK"


def test_lists_and_tensors_that_are_too_small_are_refused():
    full, short = torch.empty(B, R, C, dtype=torch.bfloat16), torch.empty(B * N - 1, dtype=torch.bfloat16)
    f32 = torch.empty(B, R, C)
    for kw in (dict(x=short), dict(out=short), dict(x=full.transpose(1, 2)), dict(x=full, ld_in=C + 1), dict(co=(1.0,) * 14),
               dict(ws=torch.empty(8, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            orth(**kw)
    for kw in (dict(grads=(full,)), dict(grads=(full, short)), dict(m=f32[:1]), dict(m_out=f32[:, 1:]), dict(w=full), dict(w_out=(f32, f32[1:])),
               dict(w_out=(f32,))):
        with pytest.raises(ValueError):
            muon(**kw)


def test_workspace_size():
    for f in (lambda *a: mrr.mrr_orthogonalize_workspace_bytes(*a), lambda *a: mrr.mrr_muon_workspace_bytes(*a)):
        assert f(0, 5, 1, "bf16") == f(5, 65537, 1, "bf16") == f(5, 5, 0, "bf16") == f(5, 5, 1, "fp8") == 0
        assert f(300, 200, 1, "f32") >= f(300, 200, 1, "bf16") > 300 * 200 * 8
        assert f(300, 200, 6, "bf16") > 5 * f(300, 200, 1, "bf16") // 2
    assert mrr.mrr_muon_workspace_bytes(300, 200, 1, "bf16", nesterov=True) >= mrr.mrr_muon_workspace_bytes(300, 200, 1, "bf16", nesterov=False) + 240000
