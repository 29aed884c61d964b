"""GPU checks of mrr_orthogonalize and mrr_muon_step against the formulas in 64 bits.

How far off a result may be is what its number formats make of it: `modelled` runs the same
steps in 64 bits and rounds where the kernel does, and its distance from the exact result is
what such roundings, in their random directions, come to.  It rounds
- what is stored: X to two f16 parts (22 bits), operands of the products to 22 or, with
  products of 11 bits, to 11, without their diagonals;
- f32 sums: a product's after every 16 terms (a matrix instruction's), and each sum and product
  of the polynomial.  Those count: at a singular value of 1, a + b x + c x^2 = 3.44 - 4.78 + 2.03
  loses a digit of its terms, so that one rounding of A's diagonal (2^-24) is 2^-24 4.78 / 0.70
  of X, seven roundings of it.
The kernel's distance is held to 4 times the model's in all, and each of its rows to 4
times the model's worst row, beside half a step of the stored type.
"""
import pytest
import torch

import allreduce_reduction_nranks_amd as mrr
from gpu_common import announce

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24
CO = (3.4445, -4.7750, 2.0315)
TINY = 1e-7


def seeded(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def gradient(g, *shape, noise=0.3):
    """A few directions beside noise."""
    k = 1 + min(shape[-2:]) // 16
    low = sum(torch.randn(*shape[:-1], 1, generator=g, device="cuda") * torch.randn(*shape[:-2], 1, shape[-1], generator=g, device="cuda")
              for _ in range(k))
    return low / k ** 0.5 + noise * torch.randn(*shape, generator=g, device="cuda")


def round_f16(x, scale):
    return (x * scale).half().double() / scale


def parts2(x, scale):
    hi = round_f16(x, scale)
    return hi + round_f16(x - hi, scale)


def exact(x, co=CO, steps=5, eps=TINY):
    x = x.double()
    x = x / (x.norm() + eps)
    if x.shape[0] > x.shape[1]:
        x = x.T.contiguous()
        return _steps(x, co, steps).T.contiguous()
    return _steps(x, co, steps)


def _steps(x, co, steps):
    for k in range(steps):
        a, b, c = co[3 * k % len(co):][:3]
        m = x @ x.T.contiguous()
        x = a * x + (b * m + c * (m @ m)) @ x
    return x


def modelled(x, two, co=CO, steps=5, eps=TINY):
    x = x.double()
    x = x / (x.norm() + eps)
    if x.shape[0] > x.shape[1]:
        return modelled_steps(x.T.contiguous(), two, co, steps).T.contiguous()
    return modelled_steps(x, two, co, steps)


def r32(x):
    return x.float().double()


def product32(x, y):
    """x y^T in f32 sums of 16 terms each."""
    total = torch.zeros(len(x), len(y), dtype=torch.float64, device="cuda")
    for k in range(0, x.shape[1], 16):
        total = r32(total + x[:, k:k + 16] @ y[:, k:k + 16].T.contiguous())
    return total


def modelled_steps(x, two, co, steps):
    part = parts2 if two else round_f16
    x = parts2(x, 8192.0)
    for k in range(steps):
        a, b, c = co[3 * k % len(co):][:3]
        xp = part(x, 8192.0)
        m = product32(xp, xp)
        d = m.diagonal().clone()
        o = part(m - torch.diag(d), 512.0)
        oo = product32(o, o)
        n = r32(r32(b * o) + r32(c * r32(oo + r32(r32(d[:, None] + d[None]) * o))))
        beta = r32(a + r32(r32(b * d) + r32(c * r32(oo.diagonal() + r32(d * d)))))
        n.fill_diagonal_(0)
        x = r32(r32(beta[:, None] * x) + product32(part(n, 64.0), xp.T.contiguous()))
        if k + 1 < steps:
            x = parts2(x, 8192.0)
    return x


def close(got, want, model, rel, what, scale=1.0):
    """got against the exact result; model: the modelled; rel: half a step of the stored type, of each value of `got`."""
    off, may = (got.double() - want).norm(dim=1), scale * (model - want).norm(dim=1)
    step = rel * want.norm(dim=1) + scale * 2.0 ** -22 * (model.norm(dim=1))
    total = float(off.norm())
    assert total <= 4 * float(may.norm()) + float(step.norm()), "%s: off by %.3g, model %.3g, step %.3g" % (
        what, total, float(may.norm()), float(step.norm()))
    bad = off > 4 * float(may.max()) + step * 1.001
    assert not bool(bad.any()), "%s: %d rows off, worst %.3g against %.3g" % (what, int(bad.sum()), float(off.max()), float(may.max()))


def orth(x, out, rows, cols, batch, t, products="auto", co=None, steps=5, eps=TINY, ld_in=None, ld_out=None, sin=None, sout=None, ws=None, **kw):
    n = mrr.mrr_orthogonalize_workspace_bytes(rows, cols, batch, t, products)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda") if ws is None else ws
    return mrr.mrr_orthogonalize(x, out, rows, cols, ld_in or cols, ld_out or cols, batch, rows * cols if sin is None else sin,
                                 rows * cols if sout is None else sout, steps, co, eps, t, products, ws, n, **kw)


SHAPES = [(1, 1, 1), (1, 70, 2), (5, 3, 1), (16, 16, 3), (64, 200, 1), (65, 130, 3), (128, 128, 2), (130, 257, 1), (257, 130, 2), (300, 300, 1),
          (520, 1601, 1), (1023, 700, 1), (300, 700, 40), (700, 300, 36)]


def is_two(rows, cols, t, products):
    return products == "f32" or (products == "auto" and t != "bf16") or min(rows, cols) <= 64


@pytest.mark.parametrize("t,products", [("bf16", "auto"), ("f16", "auto"), ("f32", "auto"), ("bf16", "f32"), ("f32", "f16")])
@pytest.mark.parametrize("rows,cols,batch", SHAPES)
def test_orthogonalize(rows, cols, batch, t, products):
    announce("orth", rows, cols, batch, t, products)
    g = seeded(rows + cols)
    x = (1e-3 * gradient(g, batch, rows, cols)).to(TYPES[t])
    out = torch.full_like(x, float("nan"))
    mrr.check(orth(x, out, rows, cols, batch, t, products))
    torch.cuda.synchronize()
    rel, two = torch.finfo(TYPES[t]).eps / 2, is_two(rows, cols, t, products)
    for k in sorted({0, batch // 2, batch - 1}):
        close(out[k], exact(x[k]), modelled(x[k], two), rel, "matrix %d" % k)


@pytest.mark.parametrize("t,n", [("bf16", 4001), ("f32", 4001)])
def test_tiles_that_the_padded_side_is_no_multiple_of(t, n):
    announce("orth large", t, n)
    g = seeded(n)
    x = gradient(g, n, n + 100, noise=0.5).to(TYPES[t])
    out = torch.full_like(x, float("nan"))
    mrr.check(orth(x, out, n, n + 100, 1, t))
    close(out, exact(x), modelled(x, t != "bf16"), torch.finfo(TYPES[t]).eps / 2, "large")


@pytest.mark.parametrize("kind", ["noise", "few directions", "steep", "one column", "equal rows"])
@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_spectra(kind, t):
    announce("orth spectra", kind, t)
    g = seeded(3)
    m, n = 200, 330
    x = torch.randn(m, n, generator=g, device="cuda")
    if kind == "few directions":
        x = gradient(g, m, n, noise=0.01)
    elif kind == "steep":
        q = torch.linalg.qr(torch.randn(m, m, generator=g, device="cuda"))[0]
        x = q @ (x * (torch.arange(1, m + 1, device="cuda") ** -1.5)[:, None])
    elif kind == "one column":
        x[:, 1:] = 0
    elif kind == "equal rows":
        x = x[:1].repeat(m, 1)
    x = x.to(TYPES[t])
    out = torch.empty_like(x)
    mrr.check(orth(x, out, m, n, 1, t))
    close(out, exact(x), modelled(x, t != "bf16"), torch.finfo(TYPES[t]).eps / 2, kind)


@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1.0, 1e18, 1e30])
def test_norms_far_from_one(scale):
    """The norm is a sum in 64 bits: squares past f32's range count."""
    announce("orth scale", scale)
    g = seeded(5)
    x = (gradient(g, 90, 140) * scale)
    out = torch.empty_like(x)
    mrr.check(orth(x, out, 90, 140, 1, "f32", eps=0.0))
    close(out, exact(x, eps=0.0), modelled(x, True, eps=0.0), 2.0 ** -24, "scale")


def test_zeros_nan_and_infinities_stay_in_their_matrix():
    announce("orth zeros")
    g = seeded(6)
    x = gradient(g, 5, 100, 150).to(torch.bfloat16)
    x[1], x[2, 7, 8], x[3, 99, 149] = 0, float("nan"), float("inf")
    out = torch.empty_like(x)
    for eps in (TINY, 0.0):
        mrr.check(orth(x, out, 100, 150, 5, "bf16", eps=eps))
        assert not bool(out[1].any()) and bool(out[2].isnan().all()) and bool(out[3].isnan().all())
        assert bool(out[0].isfinite().all()) and bool(out[4].isfinite().all())


def test_other_coefficients_and_step_counts():
    announce("orth coefficients")
    g = seeded(7)
    x = gradient(g, 100, 130)
    out = torch.empty_like(x)
    cubic = (1.5, -0.5, 0.0)
    for co, steps in ((cubic, 1), (cubic, 2), (cubic * 12, 12), ((2.0, -1.5, 0.5) * 2 + CO, 3), ((1.0, 0.0, 0.0) * 3, 3)):
        mrr.check(orth(x, out, 100, 130, 1, "f32", co=co * (1 if len(co) > 3 else steps), steps=steps))
        close(out, exact(x, co, steps), modelled(x, True, co, steps), 2.0 ** -24, "%d steps" % steps)


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(70, 150), (150, 70)])
def test_strides_slices_and_in_place(t, rows, cols):
    announce("orth strides", t, rows, cols)
    g = seeded(8)
    x = gradient(g, 3, rows, cols).to(TYPES[t])
    want = torch.empty_like(x)
    mrr.check(orth(x, want, rows, cols, 3, t))
    # matrices as column slices of one wider buffer, at odd addresses
    ld = 3 * cols + 5
    wide = torch.full((rows, ld), 7.0, dtype=TYPES[t], device="cuda")
    for k in range(3):
        wide[:, 1 + k * cols:1 + (k + 1) * cols] = x[k]
    apart = torch.full((3, rows + 2, cols + 3), 7.0, dtype=TYPES[t], device="cuda")
    mrr.check(orth(wide[:, 1:], apart, rows, cols, 3, t, ld_in=ld, sin=cols, ld_out=cols + 3, sout=(rows + 2) * (cols + 3)))
    assert torch.equal(apart[:, :rows, :cols], want)
    assert bool((apart[:, rows:] == 7.0).all()) and bool((apart[:, :, cols:] == 7.0).all())
    mrr.check(orth(wide[:, 1:], wide[:, 1:], rows, cols, 3, t, ld_in=ld, sin=cols, ld_out=ld, sout=cols))
    for k in range(3):
        assert torch.equal(wide[:, 1 + k * cols:1 + (k + 1) * cols], want[k])
    assert bool((wide[:, 0] == 7.0).all()) and bool((wide[:, 1 + 3 * cols:] == 7.0).all())
    # one matrix read for all of a batch
    same = torch.empty_like(x)
    mrr.check(orth(x, same, rows, cols, 3, t, sin=0))
    assert all(torch.equal(same[k], want[0]) for k in range(3))


def muon(grads, scale, m, m_out, mu, nesterov, w, w_out, rate, decay, rows, cols, batch, tg, tw, products="auto", ld_grad=None, ld_weight=None,
         sg=None, sw=None, ws=None, **kw):
    n = mrr.mrr_muon_workspace_bytes(rows, cols, batch, tw, products, nesterov)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda") if ws is None else ws
    return mrr.mrr_muon_step(grads, len(grads), scale, m, m_out, mu, nesterov, w, w_out, rate, decay, rows, cols, ld_grad or cols,
                             ld_weight or cols, batch, rows * cols if sg is None else sg, rows * cols if sw is None else sw, 5, None, TINY, tg,
                             tw, products, ws, n, **kw)


def check_muon(grads, scale, m, m_out, mu, nesterov, w, w_out, rate, decay, tw, two):
    gs = torch.stack([x.double() for x in grads])
    g = scale * gs.sum(0)
    old = m.double() if m is not None else torch.zeros_like(g)
    new = mu * old + g
    size = scale * gs.abs().sum(0)
    assert bool(((m_out.double() - new).abs() <= U * ((len(grads) + 3) * size + 3 * (mu * old).abs()) + 1e-45).all())
    u = g + mu * new if nesterov else new
    rel = torch.finfo(TYPES[tw]).eps / 2
    for k in range(len(u)):
        want, model = exact(u[k]), modelled(u[k], two)
        # the update is added in f32: two roundings beside the stored type's
        keep = (1 - decay) * w[k].double()
        close(w_out[k], keep - rate * want, keep - rate * model, rel + 2 * U, "weight %d" % k)


@pytest.mark.parametrize("tg,tw,products", [("bf16", "bf16", "auto"), ("bf16", "f32", "auto"), ("bf16", "f32", "f16"), ("f16", "f16", "auto"),
                                            ("f32", "f32", "auto"), ("f32", "bf16", "auto")])
@pytest.mark.parametrize("rows,cols,batch,ranks,nesterov,first", [(1, 1, 1, 1, True, True), (40, 70, 2, 2, False, False), (130, 257, 2, 3, True, False),
                                                                  (257, 130, 1, 8, True, True), (600, 390, 1, 32, False, False)])
def test_muon_step(rows, cols, batch, ranks, nesterov, first, tg, tw, products):
    announce("muon", rows, cols, batch, ranks, tg, tw, products)
    g = seeded(rows * 7 + cols)
    grads = [(gradient(g, batch, rows, cols)).to(TYPES[tg]) for _ in range(ranks)]
    m = None if first else gradient(g, batch, rows, cols)
    w = (torch.randn(batch, rows, cols, generator=g, device="cuda") / cols ** 0.5).to(TYPES[tw])
    m_out, w_out = torch.full((batch, rows, cols), 7.0, device="cuda"), [torch.empty_like(w) for _ in range(ranks)]
    mrr.check(muon(grads, 1.0 / ranks, m, m_out, 0.9, nesterov, w, w_out, 0.05, 0.01, rows, cols, batch, tg, tw, products))
    torch.cuda.synchronize()
    assert all(torch.equal(x, w_out[0]) for x in w_out)
    check_muon(grads, 1.0 / ranks, m, m_out, 0.9, nesterov, w, w_out[0], 0.05, 0.01, tw, is_two(rows, cols, tw, products))
    # the same in place, and with rows apart
    m2, w2 = (m.clone() if m is not None else torch.empty_like(m_out)), [w.clone()] + [torch.empty_like(w) for _ in range(ranks - 1)]
    mrr.check(muon(grads, 1.0 / ranks, None if first else m2, m2, 0.9, nesterov, w2[0], w2, 0.05, 0.01, rows, cols, batch, tg, tw, products))
    assert torch.equal(m2, m_out) and all(torch.equal(x, w_out[0]) for x in w2)
    gw = [torch.full((batch, rows, cols + 5), 7.0, dtype=TYPES[tg], device="cuda") for _ in grads]
    for a, b in zip(gw, grads):
        a[:, :, 2:2 + cols] = b
    wide = [torch.full((batch, rows, cols + 3), 7.0, dtype=TYPES[tw], device="cuda") for _ in range(ranks + 1)]
    wide[-1][:, :, 1:1 + cols] = w
    mw = [torch.full((batch, rows, cols + 3), 7.0, device="cuda") for _ in range(2)]
    if m is not None:
        mw[0][:, :, 1:1 + cols] = m
    cut = lambda x: x[:, :, 1:1 + cols]  # noqa: E731
    mrr.check(muon([x[:, :, 2:2 + cols] for x in gw], 1.0 / ranks, None if first else cut(mw[0]), cut(mw[1]), 0.9, nesterov, cut(wide[-1]),
                   [cut(x) for x in wide[:-1]], 0.05, 0.01, rows, cols, batch, tg, tw, products, ld_grad=cols + 5, ld_weight=cols + 3,
                   sg=rows * (cols + 5), sw=rows * (cols + 3)))
    # (the squares are summed in another order: the norm may differ in its last bit of 64)
    for x in wide[:-1]:
        assert bool((x[:, :, 0] == 7.0).all()) and bool((x[:, :, 1 + cols:] == 7.0).all())
    assert torch.equal(cut(mw[1]), m_out) and bool((mw[1][:, :, 0] == 7.0).all())
    check_muon(grads, 1.0 / ranks, m, cut(mw[1]), 0.9, nesterov, w, cut(wide[0]), 0.05, 0.01, tw, is_two(rows, cols, tw, products))


def test_graph_replays_streams_and_repeats_give_the_same_bits():
    announce("muon graph")
    g = seeded(9)
    rows, cols, ranks = 260, 390, 3
    grads = [gradient(g, 1, rows, cols).bfloat16() for _ in range(ranks)]
    w0 = (torch.randn(1, rows, cols, generator=g, device="cuda") / cols ** 0.5).bfloat16()
    n = max(mrr.mrr_muon_workspace_bytes(rows, cols, 1, "bf16"), mrr.mrr_orthogonalize_workspace_bytes(rows, cols, 1, "bf16"))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    m, w, o = torch.zeros(1, rows, cols, device="cuda"), [w0.clone() for _ in range(ranks)], torch.empty_like(w0)

    def step():
        mrr.check(muon(grads, 0.3, m, m, 0.9, True, w[0], w, 0.02, 0.0, rows, cols, 1, "bf16", "bf16", ws=ws))
        mrr.check(orth(w[1], o, rows, cols, 1, "bf16", ws=ws))

    def reset():
        m.zero_()
        for x in w:
            x.copy_(w0)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            step()
    torch.cuda.synchronize()
    want = [x.clone() for x in [m, o] + w]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        reset()
        for k in range(3):
            graph.replay()
            torch.cuda.synchronize()
            orth(grads[k].clone(), torch.empty_like(o), rows, cols, 1, "bf16")
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip([m, o] + w, want))
