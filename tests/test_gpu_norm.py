"""GPU checks of mrr_layernorm_fwd / _bwd against the formulas in 64 bits.

Tolerances, written u = 2^-24 (half a step of f32 relative to the value) and
eps/2 for half a step of the stored type:
- a stored value is off by eps/2 of itself for its one rounding;
- a sum of n terms in f32 is off by at most u times (its longest chain of
  additions) times the sum of the terms' sizes;
- a product of f32 values adds u of itself.
The oracle takes what the kernel was given (its stored h, mean, rstd), so only
the kernel's own operations count.  K bounds the chains: 16 elements a lane, 6
steps over a wave, up to 16 waves; a lane's share of a row too long for
registers is cols / 1024.
"""
import pytest
import torch

import allreduce_reduction_nranks_amd as mrr
from gpu_common import announce

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24
EPS = 1e-5


def chain(cols):
    return 64 + cols / 1024


def half_step(t):
    """Relative and absolute half step of a type."""
    f = torch.finfo(TYPES[t])
    return f.eps / 2, f.smallest_normal * f.eps / 2


def randn(g, *shape, t="f32", scale=1.0, shift=0.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale + shift).to(TYPES[t])


def seeded(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def close(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bool(bad.any()), "%s: %d of %d off, worst %.3g of the tolerance" % (
        what, int(bad.sum()), bad.numel(), float(((got.double() - want).abs() / tol).max()))


def check_forward(inputs, residual, weight, bias, h, y, mean, rstd, t, cols, eps=EPS):
    rel, sub = half_step(t)
    x = torch.stack([i.double() for i in inputs] + ([residual.double()] if residual is not None else []))
    if h is not None:
        close(h, x.sum(0), rel * x.sum(0).abs() + len(x) * U * x.abs().sum(0) + sub, "sum")
        hd = h.double()
    else:
        assert len(x) == 1
        hd = x[0]
    k = chain(cols)
    m = hd.mean(1)
    size = hd.abs().mean(1)
    var = (hd - m[:, None]).square().mean(1)
    rs = (var + eps).rsqrt()
    # an error d of the mean adds d^2 to the variance
    dm = k * U * size
    drs = rs * (k * U + dm * dm * rs * rs)
    if mean is not None:
        close(mean, m, dm + 1e-45, "mean")
        close(rstd, rs, drs, "rstd")
    w = weight.double() if weight is not None else torch.ones((), dtype=torch.float64, device="cuda")
    b = bias.double() if bias is not None else torch.zeros((), dtype=torch.float64, device="cuda")
    xhat = (hd - m[:, None]) * rs[:, None]
    want = xhat * w + b
    tol = rel * want.abs() + sub + 8 * U * ((xhat * w).abs() + b.abs()) \
        + w.abs() * ((rs * dm)[:, None] + (drs / rs)[:, None] * xhat.abs()) * (1 + rel)
    close(y, want, tol * 1.001, "out")


def forward(inputs, residual, weight, bias, h, y, mean, rstd, rows, cols, t, tw, ld_in=None, ld_out=None, eps=EPS, **kw):
    return mrr.mrr_layernorm_fwd(inputs, len(inputs), residual, weight, bias, h, y, mean, rstd, rows, cols, ld_in or cols,
                                 ld_out or cols, eps, t, tw, **kw)


SHAPES = [(1, 1), (3, 7), (5, 64), (2, 511), (9, 513), (33, 1023), (2, 1600), (3, 2049), (7, 4096), (2, 8191), (3, 16384),
          (2, 16385), (1, 70001), (1100, 96)]


@pytest.mark.parametrize("t,tw", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("ranks,res", [(1, False), (1, True), (2, False), (7, True)])
def test_forward(t, tw, rows, cols, ranks, res):
    announce("norm_fwd", t, tw, rows, cols, ranks, res)
    g = seeded(rows * 1000 + cols + ranks)
    inputs = [randn(g, rows, cols, t=t, shift=0.5) for _ in range(ranks)]
    residual = randn(g, rows, cols, t=t, scale=2.0) if res else None
    weight, bias = randn(g, cols, t=tw, shift=1.0), randn(g, cols, t=tw)
    h = torch.empty(rows, cols, dtype=TYPES[t], device="cuda") if ranks > 1 or res else None
    y = torch.full((rows, cols), float("nan"), dtype=TYPES[t], device="cuda")
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    mrr.check(forward(inputs, residual, weight, bias, h, y, mean, rstd, rows, cols, t, tw))
    torch.cuda.synchronize()
    check_forward(inputs, residual, weight, bias, h, y, mean, rstd, t, cols)


def test_forward_of_32_ranks_without_weights_or_statistics():
    announce("norm_fwd 32 ranks")
    g = seeded(5)
    inputs = [randn(g, 6, 700, t="bf16") for _ in range(32)]
    h, y = (torch.empty(6, 700, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    mrr.check(forward(inputs, None, None, None, h, y, None, None, 6, 700, "bf16", "auto"))
    check_forward(inputs, None, None, None, h, y, None, None, "bf16", 700)


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [300, 4100, 20001])
def test_strides_odd_addresses_and_rows_side_by_side(t, cols):
    announce("norm strides", t, cols)
    g = seeded(9)
    rows = 5
    wide = randn(g, rows + 1, 3 * cols + 5, t=t)
    a, b = wide[:rows, 1:1 + cols], wide[:rows, cols + 2:2 * cols + 2]
    w = randn(g, cols + 1, t=t)[1:]
    out = torch.full((rows, 2 * cols + 3), 7.0, dtype=TYPES[t], device="cuda")
    h, y = out[:, 1:1 + cols], out[:, cols + 2:2 * cols + 2]
    mrr.check(forward([a, b], None, w, None, h, y, None, None, rows, cols, t, "auto", 3 * cols + 5, 2 * cols + 3))
    check_forward([a, b], None, w, None, h, y, None, None, t, cols)
    # nothing beside the rows is written
    assert bool((out[:, 0] == 7).all()) and bool((out[:, cols + 1] == 7).all()) and bool((out[:, 2 * cols + 2] == 7).all())


@pytest.mark.parametrize("cols", [640, 20000])
def test_outputs_in_the_place_of_inputs(cols):
    announce("norm in place", cols)
    g = seeded(11)
    inputs = [randn(g, 4, cols, t="f16") for _ in range(3)]
    residual = randn(g, 4, cols, t="f16")
    want = [torch.empty_like(residual) for _ in range(2)]
    mrr.check(forward(inputs, residual, None, None, want[0], want[1], None, None, 4, cols, "f16", "auto"))
    mrr.check(forward(inputs, residual, None, None, residual, inputs[1], None, None, 4, cols, "f16", "auto"))
    assert torch.equal(residual, want[0]) and torch.equal(inputs[1], want[1])
    dout, dres = randn(g, 4, cols, t="f16"), randn(g, 4, cols, t="f16")
    mean, rstd = want[0].float().mean(1), torch.ones(4, device="cuda")
    n = mrr.mrr_layernorm_bwd_workspace_bytes(4, cols)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    got = []
    for place in (None, 0, 1, 2):
        src = [x.clone() for x in (dout, want[0], dres)]
        d = torch.empty_like(dout) if place is None else src[place]
        dw, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
        mrr.check(mrr.mrr_layernorm_bwd(src[0], src[1], None, mean, rstd, src[2], d, dw, db, 4, cols, cols, cols, "f16",
                                        "f32", ws, n))
        got.append((d, dw, db))
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))


def test_rows_that_are_constant_far_from_zero_or_not_finite():
    announce("norm special rows")
    g = seeded(13)
    x = randn(g, 7, 1000)
    x[0] = 3.0                       # no variance: y = bias
    x[1] = x[1] + 4096.0             # mean far larger than the deviation
    x[2, 5] = float("inf")
    x[3, 999] = float("nan")
    x[4] = torch.finfo(torch.float32).min
    x[5] = 0.0
    bias = randn(g, 1000)
    y = torch.empty_like(x)
    mean, rstd = torch.empty(7, device="cuda"), torch.empty(7, device="cuda")
    mrr.check(forward([x], None, None, bias, None, y, mean, rstd, 7, 1000, "f32", "f32"))
    for k in (0, 1, 5, 6):
        check_forward([x[k:k + 1]], None, None, bias, None, y[k:k + 1], mean[k:k + 1], rstd[k:k + 1], "f32", 1000)
    assert torch.equal(y[5], bias)
    assert bool(y[2].isnan().all()) and bool(y[3].isnan().all())
    assert float(mean[2]) == float("inf") and bool(mean[3].isnan())


def check_backward(dout, h, weight, mean, rstd, dres, dsum, dw, db, t, tw, rows, cols):
    rel, sub = half_step(t)
    k = chain(cols)
    dy, w = dout.double(), (weight.double() if weight is not None else torch.ones(cols, dtype=torch.float64, device="cuda"))
    rs = rstd.double()[:, None]
    xhat = (h.double() - mean.double()[:, None]) * rs
    gr = dy * w
    c1, c2 = gr.mean(1, keepdim=True), (gr * xhat).mean(1, keepdim=True)
    a1, a2 = gr.abs().mean(1, keepdim=True), (gr * xhat).abs().mean(1, keepdim=True)
    if dsum is not None:
        want = (gr - c1 - xhat * c2) * rs
        tol = U * rs * (8 * gr.abs() + (k + 8) * (a1 + xhat.abs() * a2))
        if dres is not None:
            want = want + dres.double()
            tol = tol + U * want.abs()
        close(dsum, want, (tol + rel * (want.abs() + tol) + sub) * 1.001, "dsum")
    wrel, wsub = half_step(tw)
    # a group's rows one after the other, 16 chains of groups, then those
    n = -(-rows // 256) + 1024 / 16 + 16 + 4
    if dw is not None:
        want = (dy * xhat).sum(0)
        close(dw, want, wrel * want.abs() + wsub + (n * U) * (dy * xhat).abs().sum(0) * (1 + wrel), "dweight")
    if db is not None:
        want = dy.sum(0)
        close(db, want, wrel * want.abs() + wsub + (n * U) * dy.abs().sum(0) * (1 + wrel), "dbias")


@pytest.mark.parametrize("t,tw", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("res", [False, True])
def test_backward(t, tw, rows, cols, res):
    announce("norm_bwd", t, tw, rows, cols, res)
    g = seeded(rows * 1000 + cols)
    h, dout = randn(g, rows, cols, t=t, scale=2.0, shift=0.3), randn(g, rows, cols, t=t)
    dres = randn(g, rows, cols, t=t) if res else None
    weight = randn(g, cols, t=tw, shift=1.0)
    mean, rstd = h.float().mean(1), (h.float().var(1, unbiased=False) + EPS).rsqrt()
    dsum = torch.full_like(h, float("nan"))
    dw, db = (torch.full((cols,), float("nan"), dtype=TYPES[tw], device="cuda") for _ in range(2))
    n = mrr.mrr_layernorm_bwd_workspace_bytes(rows, cols)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    mrr.check(mrr.mrr_layernorm_bwd(dout, h, weight, mean, rstd, dres, dsum, dw, db, rows, cols, cols, cols, t, tw, ws, n))
    torch.cuda.synchronize()
    check_backward(dout, h, weight, mean, rstd, dres, dsum, dw, db, t, tw, rows, cols)


@pytest.mark.parametrize("want", ["dsum", "dweight", "dbias"])
@pytest.mark.parametrize("cols", [200, 17000])
def test_backward_of_one_output_alone(want, cols):
    announce("norm_bwd alone", want, cols)
    g = seeded(17)
    h, dout = randn(g, 30, cols, t="bf16"), randn(g, 30, cols, t="bf16")
    mean, rstd = h.float().mean(1), torch.ones(30, device="cuda")
    n = mrr.mrr_layernorm_bwd_workspace_bytes(30, cols)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    o = {"dsum": torch.empty_like(h), "dweight": torch.empty(cols, device="cuda"), "dbias": torch.empty(cols, device="cuda")}
    o = {k: v if k == want else None for k, v in o.items()}
    alone = dict(workspace=None, workspace_bytes=0) if want == "dsum" else dict(workspace=ws, workspace_bytes=n)
    mrr.check(mrr.mrr_layernorm_bwd(dout, h, None, mean, rstd, None, o["dsum"], o["dweight"], o["dbias"], 30, cols, cols,
                                    cols, "bf16", "f32", **alone))
    check_backward(dout, h, None, mean, rstd, None, o["dsum"], o["dweight"], o["dbias"], "bf16", "f32", 30, cols)


def test_backward_of_no_rows_is_zero():
    announce("norm_bwd no rows")
    dw, db = torch.full((70,), 3.0, device="cuda"), torch.full((70,), 3.0, device="cuda")
    mrr.check(mrr.mrr_layernorm_bwd(None, None, None, None, None, None, None, dw, db, 0, 70, 70, 70, "bf16", "f32", None, 0))
    assert not bool(dw.any()) and not bool(db.any())


@pytest.mark.parametrize("cols", [96, 3000])
def test_gradient_is_the_slope_of_the_forward(cols):
    """<dsum, v> against (L(h + e v) - L(h - e v)) / 2e, L = <dout, y> taken in 64
    bits from the f32 kernel's y.  Each y is off by less than 64 u of its terms;
    the step's own error falls with e^2, so that of e is a third of the
    difference between the slopes at e and 2e."""
    announce("norm slope", cols)
    g = seeded(19)
    h, v, dout, w = (randn(g, 8, cols) for _ in range(4))
    w = w[0].contiguous()
    y, mean, rstd = torch.empty_like(h), torch.empty(8, device="cuda"), torch.empty(8, device="cuda")

    def loss(x):
        mrr.check(forward([x], None, w, None, None, y, mean, rstd, 8, cols, "f32", "f32"))
        return float((dout.double() * y.double()).sum())

    loss(h)
    dsum = torch.empty_like(h)
    mrr.check(mrr.mrr_layernorm_bwd(dout, h, w, mean, rstd, None, dsum, None, None, 8, cols, cols, cols, "f32", "f32"))
    slope = float((dsum.double() * v.double()).sum())
    size = float((dout.double() * y.double()).abs().sum())

    def measured(e):
        plus, minus = h + e * v, h - e * v
        # the points as they were rounded
        d = float(((plus.double() - minus.double()) * v.double()).sum() / (v.double() ** 2).sum())
        return (loss(plus) - loss(minus)) / d

    e = 2.0 ** -7
    one, two = measured(e), measured(2 * e)
    assert abs(one - slope) <= abs(two - one) + 64 * U * size / e + 1e-6 * size


def test_another_stream_and_replays_of_a_graph():
    announce("norm graph")
    g = seeded(23)
    rows, cols = 700, 1000
    x, res, dout = (randn(g, rows, cols, t="bf16") for _ in range(3))
    w = randn(g, cols)
    h, y, dsum = (torch.empty_like(x) for _ in range(3))
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dw, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    n = mrr.mrr_layernorm_bwd_workspace_bytes(rows, cols)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def step(stream=None):
        mrr.check(forward([x], res, w, None, h, y, mean, rstd, rows, cols, "bf16", "f32", stream=stream))
        mrr.check(mrr.mrr_layernorm_bwd(dout, h, w, mean, rstd, res, dsum, dw, db, rows, cols, cols, cols, "bf16", "f32",
                                        ws, n, stream=stream))
        return [o.clone() for o in (h, y, mean, rstd, dsum, dw, db)]

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(4):
        x.copy_(randn(g, rows, cols, t="bf16"))
        want = step()
        for o in (h, y, mean, rstd, dsum, dw, db):
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (h, y, mean, rstd, dsum, dw, db))), k


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1500, 1000), (1030, 1003), (1200, 4100), (1100, 4096), (1025, 8200), (1025, 8192), (40, 33000),
                                       (1024, 1600), (1024, 77), (700, 3001), (1025, 7)])
def test_backward_on_both_sides_of_the_one_launch_rule(rows, cols, t):
    """Rows that end inside a unit and whole ones, each through both ways to the weight
    gradients; with outputs in an input's place as without."""
    announce("norm_bwd ways", t, rows, cols)
    g = seeded(rows + cols)
    dout, h, dres = (randn(g, rows, cols, t=t, shift=0.1) for _ in range(3))
    weight = randn(g, cols, t="f32", shift=1.0)
    mean = h.float().mean(1)
    rstd = torch.rsqrt(h.float().var(1, unbiased=False) + EPS) if cols > 1 else torch.ones(rows, device="cuda")
    n = mrr.mrr_layernorm_bwd_workspace_bytes(rows, cols)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    first = None
    for place in (None, 0, 1, 2):
        src = [x.clone() for x in (dout, h, dres)]
        dsum = torch.full_like(h, 7.0) if place is None else src[place]
        dw, db = torch.full((cols,), 7.0, device="cuda"), torch.full((cols,), 7.0, device="cuda")
        mrr.check(mrr.mrr_layernorm_bwd(src[0], src[1], weight, mean, rstd, src[2], dsum, dw, db, rows, cols, cols, cols, t,
                                        "f32", ws, n))
        if first is None:
            first = (dsum, dw, db)
            check_backward(dout, h, weight, mean, rstd, dres, dsum, dw, db, t, "f32", rows, cols)
        assert all(torch.equal(a, b) for a, b in zip(first, (dsum, dw, db))), place


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(3, 1001), (2, 2050), (3, 4099), (2, 8197), (300, 515), (300, 2052), (40, 7)])
def test_sums_in_the_place_of_inputs_where_rows_end_inside_a_unit(rows, cols, t):
    announce("norm_fwd in place", t, rows, cols)
    g = seeded(rows + cols)
    inputs = [randn(g, rows, cols, t=t) for _ in range(3)]
    residual = randn(g, rows, cols, t=t)
    h, y = torch.empty_like(residual), torch.empty_like(residual)
    mrr.check(forward(inputs, residual, None, None, h, y, None, None, rows, cols, t, "auto"))
    for k in range(4):
        src = [x.clone() for x in inputs + [residual]]
        out = src[(k + 1) % 4]
        mrr.check(forward(src[:3], src[3], None, None, src[k], out, None, None, rows, cols, t, "auto"))
        assert torch.equal(src[k], h) and torch.equal(out, y), k


@pytest.mark.parametrize("cols", [700, 8200, 33000])
def test_rows_four_gigabytes_apart(cols):
    """All operands are columns of one buffer whose rows are 2^31 elements apart: every
    offset but the first row's passes 32 bits."""
    announce("norm far rows", cols)
    g = seeded(cols)
    rows, ld = 3, 1 << 31
    room = torch.empty((rows - 1) * ld + 8 * 33024, dtype=torch.bfloat16, device="cuda")
    view = [room.as_strided((rows, cols), (ld, 1), 33024 * k) for k in range(8)]
    for v in view[:3]:
        v.copy_(randn(g, rows, cols, t="bf16"))
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    weight = randn(g, cols, t="f32", shift=1.0)
    mrr.check(forward(view[:2], view[2], weight, None, view[3], view[4], mean, rstd, rows, cols, "bf16", "f32", ld, ld))
    check_forward(view[:2], view[2], weight, None, view[3], view[4], mean, rstd, "bf16", cols)
    n = mrr.mrr_layernorm_bwd_workspace_bytes(rows, cols)
    ws, dw, db = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    mrr.check(mrr.mrr_layernorm_bwd(view[0], view[3], weight, mean, rstd, view[1], view[5], dw, db, rows, cols, ld, ld, "bf16",
                                    "f32", ws, n))
    check_backward(view[0], view[3], weight, mean, rstd, view[1], view[5], dw, db, "bf16", "f32", rows, cols)


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(2000, 4104), (2000, 4101), (1500, 9000), (1500, 8201), (3000, 2051), (900, 2051)])
def test_gradients_in_place_of_rows_whose_last_unit_two_waves_hold(rows, cols, t):
    announce("norm_bwd in place", t, rows, cols)
    g = seeded(rows)
    src = [randn(g, rows, cols, t=t) for _ in range(3)]
    mean = src[1].float().mean(1)
    rstd = torch.rsqrt(src[1].float().var(1, unbiased=False) + EPS)
    n = mrr.mrr_layernorm_bwd_workspace_bytes(rows, cols)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    first = None
    for place in (None, 0, 1, 2, 2, 2):
        x = [v.clone() for v in src]
        dsum = torch.empty_like(x[0]) if place is None else x[place]
        dw, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
        mrr.check(mrr.mrr_layernorm_bwd(x[0], x[1], None, mean, rstd, x[2], dsum, dw, db, rows, cols, cols, cols, t, "f32", ws, n))
        first = first or (dsum, dw, db)
        assert all(torch.equal(a, b) for a, b in zip(first, (dsum, dw, db))), place
    check_backward(src[0], src[1], None, mean, rstd, src[2], *first, t, "f32", rows, cols)
