"""GPU checks of mrr_qknorm_rope_fwd / _bwd against the formulas in 64 bits.

Tolerances, u = 2^-24 (half a step of f32 relative to the value) and eps/2 for half a step of
the stored type: a stored value is off by eps/2 of itself; a sum in f32 by u times its longest
chain of additions times the sum of the terms' sizes.  A head's sum has at most 16 elements a
lane and 6 steps over a wave, so with the square, the mean, eps, the root and the quotient rs
is off by less than 16 u, an element of y by 16 u more for its two products and the rotation:
32 u of |p c| + |q s|.  The gradient adds the second sum: 64 u of its terms' sizes.  A weight's
gradient has chains of a lane's own terms (up to 128 here), 6 steps over a wave, 4 waves, 64
groups and 16 chains: 256 u.  The oracle takes the kernel's own stored h.
"""
import pytest
import torch

import allreduce_reduction_nranks_amd as mrr
from gpu_common import announce

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24
EPS = 1e-6
ROWS = 300  # of the table


def half_step(t):
    f = torch.finfo(TYPES[t])
    return f.eps / 2, f.smallest_normal * f.eps / 2


def seeded(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, t="f32", scale=1.0, shift=0.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale + shift).to(TYPES[t])


def table_of(rot, rows=ROWS):
    half = rot // 2
    f = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / max(1, half))
    a = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def close(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bool(bad.any()), "%s: %d of %d off, worst %.3g of the tolerance" % (
        what, int(bad.sum()), bad.numel(), float(((got.double() - want).abs() / tol).max()))


def turned(x, c, s, rot, pairs):
    """The rotation, and with it the sum of its terms' sizes."""
    if pairs:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        join = lambda y, z: torch.stack([y, z], -1).flatten(-2)  # noqa: E731
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        join = lambda y, z: torch.cat([y, z], -1)  # noqa: E731
    size = join((a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs())
    return torch.cat([join(a * c - b * s, b * c + a * s), x[..., rot:]], -1), torch.cat([size, x[..., rot:].abs()], -1)


def angles(table, positions, rot):
    row = table.double()[positions.clamp(min=0)][:, None]
    return row[..., :rot // 2], row[..., rot // 2:]


def check_forward(inputs, weights, table, positions, h, outs, heads, dim, rot, pairs, t):
    """outs: [tokens, heads, dim] views; rows of negative positions are not looked at."""
    rel, sub = half_step(t)
    live = positions >= 0
    x = torch.stack([i.double() for i in inputs])
    if h is None:
        hd = x.sum(0)
        if len(inputs) > 1:
            hd = hd.to(TYPES[t]).double()  # (only where the f32 sum is exact, or of one rank)
    else:
        close(h[live], x.sum(0)[live], (rel * x.sum(0).abs() + len(inputs) * U * x.abs().sum(0) + sub)[live], "sum")
        hd = h.double()
    c, s = angles(table, positions, rot)
    first = 0
    for k, n in enumerate(heads):
        p = hd[:, first * dim:(first + n) * dim].reshape(len(hd), n, dim)
        first += n
        if outs[k] is None or not n:
            continue
        if k == 2:
            assert torch.equal(outs[k][live].double(), p[live])
            continue
        w = weights[k].double() if weights[k] is not None else 1.0
        y, size = turned(p * torch.rsqrt(p.square().mean(-1, keepdim=True) + EPS) * w, c, s, rot, pairs)
        close(outs[k][live], y[live], (rel * y.abs() + 32 * U * size + sub)[live], "qk"[k])


def forward(inputs, weights, table, positions, h, outs, heads, dim, rot, pairs, t, tw, ld_in=None, lds=None, strides=None, tokens=None,
            **kw):
    return mrr.mrr_qknorm_rope_fwd(inputs, len(inputs), weights[0], weights[1], table, table.shape[0], positions, h, outs,
                                   len(inputs[0]) if tokens is None else tokens, heads, dim, rot, pairs, ld_in or sum(heads) * dim,
                                   lds or [n * dim for n in heads], strides or [dim] * 3, EPS, t, tw, **kw)


def empty_outs(tokens, heads, dim, t):
    return [torch.full((tokens, n, dim), 7.0, dtype=TYPES[t], device="cuda") for n in heads]


# tokens, heads, head elements, rotated: whole vectors, heads that end inside one, parts shorter than one, one element
SHAPES = [(1, (32, 8, 8), 128, 128), (5, (3, 1, 2), 64, 64), (70, (2, 2, 0), 80, 32), (9, (7, 1, 1), 96, 48), (33, (1, 1, 1), 53, 26),
          (4, (2, 1, 1), 1, 0), (3, (2, 3, 1), 2, 2), (6, (1, 0, 1), 20, 10), (11, (2, 1, 1), 68, 64), (3, (2, 1, 0), 512, 512),
          (2, (1, 2, 1), 511, 510), (2, (2, 1, 1), 500, 6), (2, (1, 1, 1), 256, 0), (1030, (5, 2, 1), 32, 16), (2, (3, 0, 0), 172, 86)]


@pytest.mark.parametrize("t,tw", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("tokens,heads,dim,rot", SHAPES)
@pytest.mark.parametrize("ranks", [1, 5])
def test_forward(t, tw, pairs, tokens, heads, dim, rot, ranks):
    announce("qk_fwd", t, tw, pairs, tokens, heads, dim, rot, ranks)
    g = seeded(tokens * 100 + dim + ranks)
    width = sum(heads) * dim
    inputs = [randn(g, tokens, width, t=t, shift=0.1) for _ in range(ranks)]
    weights = [randn(g, dim, t=tw, shift=1.0) for _ in range(2)]
    positions = torch.randint(0, ROWS, (tokens,), generator=g, device="cuda")
    positions[torch.rand(tokens, generator=g, device="cuda") < 0.2] = -1
    h = torch.full((tokens, width), 7.0, dtype=TYPES[t], device="cuda") if ranks > 1 else None
    outs = empty_outs(tokens, heads, dim, t)
    mrr.check(forward(inputs, weights, table_of(rot), positions, h, outs, list(heads), dim, rot, pairs, t, tw))
    torch.cuda.synchronize()
    check_forward(inputs, weights, table_of(rot), positions, h, outs, heads, dim, rot, pairs, t)
    # a padded token's rows are left as they were
    for o in outs + ([h] if h is not None else []):
        assert bool((o[positions < 0] == 7.0).all())


def backward_tolerances(douts, h, weights, table, positions, heads, dim, rot, pairs, t):
    """Expected gradients and what each may be off by."""
    rel, sub = half_step(t)
    live = (positions >= 0)[:, None, None]
    c, s = angles(table, positions, rot)
    hd = h.double().view(len(h), -1, dim)
    want, tol, dw, tw = [], [], [], []
    first = 0
    for k, n in enumerate(heads):
        x = hd[:, first:first + n]
        first += n
        dy = douts[k].double() if douts[k] is not None else torch.zeros_like(x)
        dy = torch.where(live, dy, 0.0)
        if k == 2:
            want.append(dy)
            tol.append(torch.zeros_like(dy))
            continue
        w = weights[k].double() if weights[k] is not None else torch.ones((), dtype=torch.float64, device="cuda")
        x = torch.where(live, x, 1.0)
        rs = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        u, size = turned(dy, c, -s, rot, pairs)
        xh = x * rs
        d = rs * (u * w - xh * (u * w * xh).mean(-1, keepdim=True))
        bound = rs * (size * w.abs() + xh.abs() * (size * w.abs() * xh.abs()).mean(-1, keepdim=True))
        want.append(d)
        tol.append(rel * d.abs() + 64 * U * bound + sub)
        dw.append((u * xh).sum((0, 1)))
        tw.append((256 * U * size * xh.abs()).sum((0, 1)))
    return torch.cat(want, 1).flatten(1), torch.cat(tol, 1).flatten(1), dw, tw


def backward(douts, h, weights, table, positions, dsum, dws, heads, dim, rot, pairs, t, tw, ld_in=None, lds=None, strides=None, ws=None, **kw):
    n = mrr.mrr_qknorm_rope_bwd_workspace_bytes(len(h), heads, dim)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda") if ws is None else ws
    return mrr.mrr_qknorm_rope_bwd(douts, h, weights[0], weights[1], table, table.shape[0], positions, dsum, dws[0], dws[1], len(h), heads,
                                   dim, rot, pairs, ld_in or sum(heads) * dim, lds or [n * dim for n in heads], strides or [dim] * 3,
                                   EPS, t, tw, ws, n, **kw)


def check_backward(douts, h, weights, table, positions, dsum, dws, heads, dim, rot, pairs, t, tw):
    want, tol, dw, tdw = backward_tolerances(douts, h, weights, table, positions, heads, dim, rot, pairs, t)
    if dsum is not None:
        close(dsum, want, tol, "dsum")
    rel, sub = half_step(tw)
    for k in range(2):
        if dws[k] is not None:
            close(dws[k], dw[k], rel * dw[k].abs() + tdw[k] * (1 + rel) + sub, "d%s_weight" % "qk"[k])


@pytest.mark.parametrize("t,tw", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("tokens,heads,dim,rot", SHAPES + [(4500, (2, 1, 1), 64, 32)])
def test_backward(t, tw, pairs, tokens, heads, dim, rot):
    announce("qk_bwd", t, tw, pairs, tokens, heads, dim, rot)
    g = seeded(tokens * 100 + dim)
    width = sum(heads) * dim
    h = randn(g, tokens, width, t=t, shift=0.1)
    weights = [randn(g, dim, t=tw, shift=1.0) for _ in range(2)]
    positions = torch.randint(0, ROWS, (tokens,), generator=g, device="cuda")
    positions[torch.rand(tokens, generator=g, device="cuda") < 0.2] = -3
    douts = [randn(g, tokens, n, dim, t=t) for n in heads]
    h[positions < 0] = float("nan")  # not read
    for d in douts:
        d[positions < 0] = float("inf")
    dsum = torch.full((tokens, width), 7.0, dtype=TYPES[t], device="cuda")
    dws = [torch.full((dim,), 7.0, dtype=TYPES[tw], device="cuda") for _ in range(2)]
    table = table_of(rot)
    mrr.check(backward(douts, h, weights, table, positions, dsum, dws, list(heads), dim, rot, pairs, t, tw))
    torch.cuda.synchronize()
    check_backward(douts, h, weights, table, positions, dsum, dws, heads, dim, rot, pairs, t, tw)
    assert not bool(dsum[positions < 0].any())


@pytest.mark.parametrize("pairs", [False, True])
def test_gradients_are_differences_of_the_forward(pairs):
    """f32: a step of e along v changes the weighted sum of the outputs by e times the gradient's product with v, up to e^2 (the
    second derivative) and the outputs' own rounding."""
    announce("qk differences", pairs)
    tokens, heads, dim, rot = 6, [3, 2, 1], 24, 16
    g = seeded(4)
    h, table = randn(g, tokens, sum(heads) * dim), table_of(rot)
    weights = [randn(g, dim, shift=1.0) for _ in range(2)]
    positions = torch.arange(tokens, device="cuda") * 7
    douts = [randn(g, tokens, n, dim) for n in heads]
    dsum, dws = torch.empty_like(h), [torch.empty(dim, device="cuda") for _ in range(2)]
    mrr.check(backward(douts, h, weights, table, positions, dsum, dws, heads, dim, rot, pairs, "f32", "f32"))

    def value(x, w):
        outs = empty_outs(tokens, heads, dim, "f32")
        mrr.check(forward([x], w, table, positions, None, outs, heads, dim, rot, pairs, "f32", "f32"))
        return sum(float((o.double() * d.double()).sum()) for o, d in zip(outs, douts))

    v, vw = randn(g, *h.shape), [randn(g, dim) for _ in range(2)]
    e = 2.0 ** -8
    step = value(h + e * v, [w + e * d for w, d in zip(weights, vw)]) - value(h - e * v, [w - e * d for w, d in zip(weights, vw)])
    want = float((dsum.double() * v.double()).sum()) + sum(float((a.double() * b.double()).sum()) for a, b in zip(dws, vw))
    size = sum(float((d.double().abs()).sum()) for d in douts)
    assert abs(step / (2 * e) - want) <= size * (8 * e * e + 64 * U / e)


@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_strides_head_by_head_and_columns_of_wider_buffers(t):
    announce("qk strides", t)
    g = seeded(8)
    tokens, heads, dim, rot = 37, [4, 2, 2], 48, 24
    width = sum(heads) * dim
    wide = randn(g, tokens, width + 11, t=t)
    x = wide[:, 5:5 + width]
    weights, table = [randn(g, dim, t=t), None], table_of(rot)
    # queries head by head, keys and values beside each other in one buffer at odd places
    q = torch.full((heads[0], tokens + 3, dim), 7.0, dtype=TYPES[t], device="cuda")
    kv = torch.full((tokens, (heads[1] + heads[2]) * dim + 3), 7.0, dtype=TYPES[t], device="cuda")
    k, v = kv[:, 1:1 + heads[1] * dim], kv[:, 2 + heads[1] * dim:2 + (heads[1] + heads[2]) * dim]
    lds, strides = [dim, kv.shape[1], kv.shape[1]], [(tokens + 3) * dim, dim, dim]
    mrr.check(forward([x], weights, table, None, None, [q, k, v], heads, dim, rot, False, t, "auto", ld_in=width + 11, lds=lds, strides=strides))
    outs = [q[:, :tokens].transpose(0, 1), k.view(tokens, heads[1], dim), v.view(tokens, heads[2], dim)]
    positions = torch.arange(tokens, device="cuda")
    check_forward([x], weights, table, positions, None, outs, heads, dim, rot, False, t)
    assert bool((q[:, tokens:] == 7.0).all()) and bool((kv[:, 0] == 7.0).all())
    assert bool((kv[:, 1 + heads[1] * dim] == 7.0).all()) and bool((kv[:, -1] == 7.0).all())
    # the same places hold the gradients backwards
    dq, dkv = randn(g, *q.shape, t=t), randn(g, *kv.shape, t=t)
    dk, dv = dkv[:, 1:1 + heads[1] * dim], dkv[:, 2 + heads[1] * dim:2 + (heads[1] + heads[2]) * dim]
    dx = torch.full((tokens, width + 11), 7.0, dtype=TYPES[t], device="cuda")
    dws = [torch.empty(dim, dtype=TYPES[t], device="cuda") for _ in range(2)]
    mrr.check(backward([dq, dk, dv], x, weights, table, None, dx[:, 5:5 + width], dws, heads, dim, rot, False, t, "auto", ld_in=width + 11,
                       lds=lds, strides=strides))
    douts = [dq[:, :tokens].transpose(0, 1), dk.view(tokens, heads[1], dim), dv.view(tokens, heads[2], dim)]
    check_backward(douts, x.contiguous(), weights, table, positions, dx[:, 5:5 + width], dws, heads, dim, rot, False, t, t)
    assert bool((dx[:, :5] == 7.0).all()) and bool((dx[:, 5 + width:] == 7.0).all())


@pytest.mark.parametrize("t", ["f16", "f32"])
@pytest.mark.parametrize("dim,rot", [(128, 128), (53, 26)])
@pytest.mark.parametrize("pairs", [False, True])
def test_in_the_place_of_the_input(t, dim, rot, pairs):
    announce("qk in place", t, dim, pairs)
    g = seeded(11)
    tokens, heads = 150, [5, 2, 3]
    a, b = (randn(g, tokens, sum(heads) * dim, t=t) for _ in range(2))
    weights, table = [randn(g, dim, t=t), randn(g, dim, t=t)], table_of(rot)
    want = empty_outs(tokens, heads, dim, t)
    mrr.check(forward([a, b], weights, table, None, None, want, heads, dim, rot, pairs, t, "auto"))
    parts, width = list(b.split([n * dim for n in heads], 1)), sum(heads) * dim
    mrr.check(forward([a, b], weights, table, None, None, parts, heads, dim, rot, pairs, t, "auto", lds=[width] * 3))
    assert torch.equal(b, torch.cat([o.flatten(1) for o in want], 1))
    # and the gradient in the place of the sum
    h, douts = randn(g, tokens, width, t=t), [randn(g, tokens, n, dim, t=t) for n in heads]
    dsum, dws = torch.empty_like(h), [torch.empty(dim, dtype=TYPES[t], device="cuda") for _ in range(2)]
    mrr.check(backward(douts, h, weights, table, None, dsum, dws, heads, dim, rot, pairs, t, "auto"))
    mrr.check(backward(douts, h, weights, table, None, h, [None, None], heads, dim, rot, pairs, t, "auto"))
    assert torch.equal(h, dsum)


def test_outputs_that_are_not_wanted():
    announce("qk outputs")
    g = seeded(12)
    tokens, heads, dim, rot = 20, [2, 2, 2], 64, 64
    h, table = randn(g, tokens, 6 * dim, t="bf16"), table_of(rot)
    weights = [randn(g, dim), randn(g, dim)]
    full = empty_outs(tokens, heads, dim, "bf16")
    mrr.check(forward([h], weights, table, None, None, full, heads, dim, rot, False, "bf16", "f32"))
    for k in range(3):
        one = [None] * 3
        one[k] = torch.full_like(full[k], 7.0)
        mrr.check(forward([h], weights, table, None, None, one, heads, dim, rot, False, "bf16", "f32"))
        assert torch.equal(one[k], full[k])
    total = torch.empty_like(h)
    mrr.check(forward([h], weights, table, None, total, [None] * 3, heads, dim, rot, False, "bf16", "f32"))
    assert torch.equal(total, h)
    positions = torch.arange(tokens, device="cuda")
    for k in range(3):
        douts = [randn(g, tokens, 2, dim, t="bf16") for _ in range(3)]
        douts[k] = None
        dsum, dws = torch.full_like(h, 7.0), [torch.full((dim,), 7.0, device="cuda") for _ in range(2)]
        mrr.check(backward(douts, h, weights, table, None, dsum, dws, heads, dim, rot, False, "bf16", "f32"))
        check_backward(douts, h, weights, table, positions, dsum, dws, heads, dim, rot, False, "bf16", "f32")
        only = [torch.full((dim,), 7.0, device="cuda"), None]
        mrr.check(backward(douts, h, weights, table, None, None, only, heads, dim, rot, False, "bf16", "f32"))
        assert torch.equal(only[0], dws[0])


def test_no_tokens_positions_past_the_table_and_values_that_are_not_finite():
    announce("qk borders")
    g = seeded(13)
    heads, dim, rot = [2, 1, 1], 64, 32
    table, weights = table_of(rot), [None, None]
    dws = [torch.full((dim,), 7.0, device="cuda") for _ in range(2)]
    mrr.check(backward([None] * 3, torch.empty(0, 4 * dim, device="cuda"), weights, table, None, None, dws, heads, dim, rot, False, "f32", "f32"))
    assert not any(bool(d.any()) for d in dws)
    h = randn(g, 4, 4 * dim)
    positions = torch.tensor([3, ROWS, ROWS - 1, 1 << 40], device="cuda")
    h[2, 5], h[0, 2 * dim + 1] = float("nan"), float("inf")
    outs = empty_outs(4, heads, dim, "f32")
    mrr.check(forward([h], weights, table, positions, None, outs, heads, dim, rot, False, "f32", "f32"))
    q, k, v = outs
    for t in (1, 3):
        assert bool(q[t, :, :rot].isnan().all()) and bool(q[t, :, rot:].isfinite().all()) and bool(k[t, :, :rot].isnan().all())
    assert bool(q[2, 0].isnan().all()) and bool(q[2, 1].isfinite().all()) and bool(k[2].isfinite().all())
    assert bool(q[0].isfinite().all()) and bool(k[0, 0, 1].isnan()) and torch.equal(v[:, 0], h[:, 3 * dim:])
    # a head of zeros
    zero = torch.zeros(2, 4 * dim, device="cuda")
    outs = empty_outs(2, heads, dim, "f32")
    mrr.check(forward([zero], weights, table, None, None, outs, heads, dim, rot, False, "f32", "f32"))
    assert not any(bool(o.any()) for o in outs)


@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_graph_replays_streams_and_repeats_give_the_same_bits(t):
    announce("qk graph", t)
    g = seeded(14)
    tokens, heads, dim, rot = 301, [6, 2, 2], 128, 64
    h, other = (randn(g, tokens, 10 * dim, t=t) for _ in range(2))
    table, weights = table_of(rot, 512), [randn(g, dim), randn(g, dim)]
    tw = "f32"
    douts = [randn(g, tokens, n, dim, t=t) for n in heads]
    ws = torch.empty(mrr.mrr_qknorm_rope_bwd_workspace_bytes(tokens, heads, dim), dtype=torch.uint8, device="cuda")
    x = h.clone()
    outs, total, dsum = empty_outs(tokens, heads, dim, t), torch.empty_like(h), torch.empty_like(h)
    dws = [torch.empty(dim, device="cuda") for _ in range(2)]

    def both():
        mrr.check(forward([x, other], weights, table, None, total, outs, heads, dim, rot, True, t, tw))
        mrr.check(backward(douts, total, weights, table, None, dsum, dws, heads, dim, rot, True, t, tw, ws=ws))

    def results():
        torch.cuda.synchronize()
        return [o.clone() for o in outs + [total, dsum] + dws]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    first = results()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for k in range(3):
        x.copy_(h if k != 1 else other)
        both()
        want = results()
        for o in outs + [total, dsum] + dws:
            o.zero_()
        graph.replay()
        got = results()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        if k != 1:
            assert all(torch.equal(a, b) for a, b in zip(got, first))
