"""GPU checks of mrr_linear_xent_fwd / _bwd against the formulas in 64 bits.

Tolerances, with u = 2^-24 (half a step of f32 relative to the value) and eps/2
for half a step of the stored type:
- a logit is a sum of C exact products, off by at most its count of terms times u
  times the sum of their sizes.  f32: of 3 C products of f16 parts, which leave out
  3 x 2^-22 of each product, and parts of an element no smaller than 2^-40 of the
  tensor's largest;
- exp is off by 2 u and by what its argument's rounding makes of it, u per unit of
  the argument on the way in (twice: the product with log2 e, its constant);
- lse moves by the logits' errors weighted with p, by the chain of its sum (64 in a
  lane, the join's 64 chains, a share of the tiles) and by its own rounding;
- dz takes half a step of its type (f16: half of its smallest step times the scale
  that is taken out again as well; f32: 2^-24, its three parts hold 24 bits);
- a gradient is off by its terms' errors, by u times its count of terms times their
  sizes, and by half a step for its rounding.
"""
import pytest
import torch

import allreduce_reduction_nranks_amd as mrr
from gpu_common import announce

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24
IGNORE = -100


def seeded(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def half_step(t):
    f = torch.finfo(TYPES[t])
    return f.eps / 2, f.smallest_normal * f.eps / 2


def close(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bool(bad.any()), "%s: %d of %d off, worst %.3g of the tolerance" % (
        what, int(bad.sum()), bad.numel(), float(((got.double() - want).abs() / tol).max()))


class Case:
    """Operands of a call, and the exact results with their tolerances."""

    def __init__(self, tokens, rows, cols, t, seed, ignored=0.2, scale=3.0, pad=0, off=0, spread=1.0):
        g = seeded(seed)
        self.tokens, self.rows, self.cols, self.t = tokens, rows, cols, t
        self.ld = cols + pad
        n = lambda *s: torch.randn(*s, generator=g, device="cuda")
        room = n(tokens * self.ld + off).mul(spread).to(TYPES[t])
        self.hidden = room[off:].view(tokens, self.ld)[:, :cols]
        self.weights = [(n(r * self.ld + off) * (scale / cols ** 0.5)).to(TYPES[t])[off:].view(r, self.ld)[:, :cols] for r in rows]
        vocab = sum(rows)
        self.targets = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
        self.targets[torch.rand(tokens, generator=g, device="cuda") < ignored] = IGNORE
        self.dloss = 0.5 + torch.rand(tokens, generator=g, device="cuda")

    def exact(self, lse=None, dloss=None):
        h, w = self.hidden.double(), torch.cat([x.double() for x in self.weights])
        f32 = self.t == "f32"
        terms = self.cols * 3 + 12 if f32 else self.cols
        z = h @ w.T
        ez = terms * U * (h.abs() @ w.abs().T)
        if f32:
            ez = ez + 2.0 ** -40 * (h.abs().sum(1)[:, None] * w.abs().max() + w.abs().sum(1)[None] * h.abs().max())
        self.lse = torch.logsumexp(z, 1)
        p = (z - self.lse[:, None]).exp()
        size = (p * z.abs()).sum(1) + z.abs().amax(1)
        vocab = z.shape[1]
        elser = (p * ez).sum(1) + U * (4 * size + 256 + vocab / 64 / 64 + 4 * self.lse.abs())
        self.elser = elser * 1.01 + ez.amax(1) ** 2
        counted = (self.targets >= 0) & (self.targets < vocab)
        at = self.targets.clamp(0, vocab - 1)[:, None]
        zt, ezt = z.gather(1, at)[:, 0], ez.gather(1, at)[:, 0]
        self.loss = torch.where(counted, self.lse - zt, 0.0)
        self.eloss = torch.where(counted, self.elser + ezt + U * (self.lse - zt).abs(), 0.0)
        if dloss is None:
            return
        dl = torch.where(counted, dloss.double().expand(self.tokens), 0.0)
        x = z - lse.double()[:, None]
        p = x.exp()
        ep = p * ((ez + U * (4 * x.abs() + 2)).exp() - 1)
        hit = torch.zeros_like(p).scatter_(1, at, 1.0) * counted[:, None]
        dz = (p - hit) * dl[:, None]
        rel, sub = half_step(self.t)
        if f32:
            rel, sub = 2.0 ** -22, half_step("f16")[1]
        sub = sub * 2 ** -13 * float(dl.abs().max()) if self.t != "bf16" else 0.0
        edz = (ep + 2 * U) * dl.abs()[:, None]
        edz = edz + rel * (dz.abs() + edz) + sub * counted[:, None]
        orel, osub = half_step(self.t)

        def grad(want, e):
            return want, (e + orel * (want.abs() + e) + osub) * 1.01

        # f32: as for a logit; a gradient left to one piece at a time adds the pieces too
        n, part = (3, 2.0 ** -40) if f32 else (1, 0.0)
        self.dhidden = grad(dz @ w, edz @ w.abs() + U * (n * vocab + 256) * (dz.abs() @ w.abs())
                            + part * w.abs().max() * dz.abs().sum(1)[:, None])
        dw, edw = grad(dz.T.contiguous() @ h, edz.T.contiguous() @ h.abs()
                       + U * (n * self.tokens + 64) * (dz.abs().T.contiguous() @ h.abs())
                       + part * h.abs().max() * dz.abs().sum(0)[:, None])
        self.dweights = list(zip(dw.split(self.rows), edw.split(self.rows)))

    def workspace(self, backward):
        n = mrr.mrr_linear_xent_workspace_bytes(self.tokens, self.cols, self.rows, len(self.rows), self.t, backward)
        return torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device="cuda"), n

    def forward(self, loss=True, lse=True, stream=None, ws=None):
        self.got_loss = torch.full((self.tokens,), 7.0, device="cuda") if loss is True else loss
        self.got_lse = torch.full((self.tokens,), 7.0, device="cuda") if lse is True else lse
        ws, n = ws or self.workspace(False)
        mrr.check(mrr.mrr_linear_xent_fwd(self.hidden, self.weights, self.rows, len(self.rows), self.targets, IGNORE,
                                          self.got_loss, self.got_lse, self.tokens, self.cols, self.ld, self.ld, self.t, ws,
                                          n, stream=stream))

    def backward(self, lse, dloss, stride=1, dhidden=True, dweights=True, stream=None, ws=None):
        def like(x):  # a buffer with the operand's strides, its gaps marked
            room = torch.full((x.shape[0] * self.ld + 8,), 7.0, dtype=TYPES[self.t], device="cuda")
            return room[:x.shape[0] * self.ld].view(-1, self.ld)[:, :self.cols]
        self.got_dh = like(self.hidden) if dhidden is True else dhidden
        self.got_dw = [like(w) for w in self.weights] if dweights is True else dweights
        ws, n = ws or self.workspace(True)
        mrr.check(mrr.mrr_linear_xent_bwd(self.hidden, self.weights, self.rows, len(self.rows), self.targets, IGNORE, lse,
                                          dloss, stride, self.got_dh, self.got_dw, self.tokens, self.cols, self.ld, self.ld,
                                          self.t, ws, n, stream=stream))

    def check_forward(self):
        self.exact()
        close(self.got_lse, self.lse, self.elser, "lse")
        close(self.got_loss, self.loss, self.eloss, "loss")

    def check_backward(self):
        if self.got_dh is not None:
            close(self.got_dh, *self.dhidden, "dhidden")
        for r, got in enumerate(self.got_dw or []):
            if got is not None and self.rows[r]:
                close(got, *self.dweights[r], "dweights[%d]" % r)


SHAPES = [
    (1, [1], 1), (1, [300], 64), (2, [5, 0, 3], 7), (1, [1000, 999], 520), (16, [257], 128), (17, [64, 64, 64], 96),
    (33, [511, 2, 700], 192), (64, [1024], 320), (65, [130, 257], 72), (127, [256], 64), (128, [512, 255], 1023),
    (129, [1, 1, 1, 1], 64), (200, [256, 256, 300], 640), (257, [1500], 257), (300, [40, 0, 600, 77], 200),
    (513, [2048, 1023], 384), (1000, [513], 1600),
]


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("tokens,rows,cols", SHAPES)
def test_forward_and_backward(tokens, rows, cols, t):
    announce("xent", t, tokens, rows, cols)
    c = Case(tokens, rows, cols, t, tokens + cols)
    c.forward()
    torch.cuda.synchronize()
    c.check_forward()
    announce("xent bwd", t, tokens, rows, cols)
    lse = c.lse.float()
    c.backward(lse, c.dloss)
    torch.cuda.synchronize()
    c.exact(lse, c.dloss)
    c.check_backward()


@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_more_than_one_piece_of_the_vocabulary(t):
    tokens, rows, cols = (2600, [30000, 35001], 64) if t == "bf16" else (1100, [50001, 20000], 64)
    announce("xent pieces", t, tokens, rows, cols)
    c = Case(tokens, rows, cols, t, 3)
    c.forward()
    torch.cuda.synchronize()
    c.check_forward()
    lse = c.lse.float()
    c.backward(lse, c.dloss)
    torch.cuda.synchronize()
    c.exact(lse, c.dloss)
    c.check_backward()


def test_laid_out_weights_of_more_than_one_piece():
    announce("xent laid out pieces")
    c = Case(20, [9000, 26000], 4095, "bf16", 4)
    c.forward()
    torch.cuda.synchronize()
    c.check_forward()
    lse = c.lse.float()
    c.backward(lse, c.dloss)
    torch.cuda.synchronize()
    c.exact(lse, c.dloss)
    c.check_backward()


@pytest.mark.parametrize("pad,off", [(8, 8), (3, 1), (64, 0), (0, 1)])
@pytest.mark.parametrize("tokens", [5, 40, 300])
@pytest.mark.parametrize("t", ["f16", "f32"])
def test_strides_and_odd_addresses(pad, off, tokens, t):
    announce("xent strides", pad, off, tokens, t)
    c = Case(tokens, [300, 77], 128, t, 5, pad=pad, off=off)
    c.forward()
    c.check_forward()
    lse = c.lse.float()
    c.backward(lse, c.dloss)
    torch.cuda.synchronize()
    c.exact(lse, c.dloss)
    c.check_backward()
    if pad:  # nothing beside the rows is written
        for x in [c.got_dh] + c.got_dw:
            rows = x.shape[0]
            assert bool((x.as_strided((rows, pad), (c.ld, 1), x.storage_offset() + 128) == 7).all())


@pytest.mark.parametrize("tokens", [1, 9, 60, 300])
def test_tokens_without_a_loss(tokens):
    """All ignored, a NaN row that is ignored, and targets outside the vocabulary."""
    announce("xent ignored", tokens)
    c = Case(tokens, [100, 200], 64, "bf16", 6, ignored=2.0)
    c.forward()
    c.check_forward()
    assert not bool(c.got_loss.any())
    lse = c.lse.float()
    c.hidden[tokens // 2] = float("nan")
    c.backward(lse, c.dloss)
    torch.cuda.synchronize()
    assert not bool(c.got_dh.any()) and not any(bool(w.any()) for w in c.got_dw)
    if tokens == 1:
        return
    c = Case(tokens, [100, 200], 64, "bf16", 7, ignored=0.3)
    c.targets[0], c.targets[tokens - 1] = 300, -1
    c.forward()
    lse = c.got_lse.clone()
    assert bool(c.got_loss[[0, tokens - 1]].isnan().all())
    c.got_loss[[0, tokens - 1]] = 0.0
    c.check_forward()
    c.exact(lse, c.dloss)
    c.hidden[0], c.hidden[tokens - 1] = float("nan"), float("inf")
    c.dloss[0] = float("nan")
    c.backward(lse, c.dloss)
    torch.cuda.synchronize()
    c.check_backward()
    assert not bool(c.got_dh[0].any()) and not bool(c.got_dh[tokens - 1].any())


@pytest.mark.parametrize("tokens", [5, 140])
def test_an_ignored_token_does_not_set_the_scale_of_f32_parts(tokens):
    announce("xent f32 scale", tokens)
    c = Case(tokens, [300, 41], 72, "f32", 30, ignored=0.0)
    c.targets[1] = IGNORE
    c.hidden[1] = 0.0
    c.exact()
    lse = c.lse.float()
    c.exact(lse, c.dloss)
    c.hidden[1] = 3e30
    c.backward(lse, c.dloss)
    torch.cuda.synchronize()
    c.check_backward()


@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_rows_in_both_sizes_of_tile(t):
    """Full rounds of large tiles and the rest in small ones, in each product."""
    tokens, rows, cols = (700, [30000, 10257], 128) if t == "bf16" else (700, [23000], 128)
    announce("xent both tiles", t)
    c = Case(tokens, rows, cols, t, 31)
    c.forward()
    torch.cuda.synchronize()
    c.check_forward()
    lse = c.lse.float()
    c.backward(lse, c.dloss)
    torch.cuda.synchronize()
    c.exact(lse, c.dloss)
    c.check_backward()


@pytest.mark.parametrize("tokens", [3, 50, 200])
@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_logits_that_are_large_or_not_finite(tokens, t):
    announce("xent special logits", tokens, t)
    # exp of these overflows without the running maximum
    c = Case(tokens, [300], 64, t, 8, spread=60.0)
    c.forward()
    c.check_forward()
    # a row of -inf weights against positive hidden states: probability 0
    c = Case(tokens, [300, 20], 64, t, 9)
    c.hidden.abs_().add_(0.1)
    c.weights[0][5] = -float("inf")
    c.weights[1][:] = -float("inf")
    c.targets.remainder_(5)
    c.forward()
    z = c.hidden.double() @ torch.cat(c.weights).double().T
    want = torch.logsumexp(z, 1)
    assert bool(((c.got_lse.double() - want).abs() <= 1e-4 * want.abs().clamp(min=1.0)).all())
    # a NaN hidden state makes its own token NaN alone
    c = Case(tokens, [300], 64, t, 10)
    c.hidden[1, 3] = float("nan")
    c.forward()
    others = [k for k in range(tokens) if k != 1]
    assert bool(c.got_lse[1].isnan()) and bool(c.got_lse[others].isfinite().all())


@pytest.mark.parametrize("tokens", [6, 70])
@pytest.mark.parametrize("t", ["f16", "bf16", "f32"])
def test_one_gradient_for_all_and_small_or_large_ones(tokens, t):
    announce("xent dloss", tokens, t)
    c = Case(tokens, [400, 300], 64, t, 11)
    c.exact()
    lse = c.lse.float()
    one = torch.full((1,), 1.0 / tokens, device="cuda")
    c.backward(lse, one, stride=0)
    c.exact(lse, one)
    c.check_backward()
    apart = torch.rand(tokens, 5, device="cuda", generator=seeded(1))
    c.backward(lse, apart, stride=5)
    c.exact(lse, apart[:, 0])
    c.check_backward()
    for scale in (1e-6, 2e3, 0.0):
        d = c.dloss * scale
        c.backward(lse, d)
        c.exact(lse, d)
        c.check_backward()


@pytest.mark.parametrize("tokens", [4, 150])
def test_some_outputs_alone_and_in_place(tokens):
    announce("xent alone", tokens)
    c = Case(tokens, [300, 50, 70], 128, "bf16", 12)
    c.forward()
    both = c.got_loss.clone(), c.got_lse.clone()
    c.forward(loss=None)
    assert torch.equal(c.got_lse, both[1])
    c.forward(lse=None)
    assert torch.equal(c.got_loss, both[0])
    lse = both[1]
    c.backward(lse, c.dloss)
    dh, dw = c.got_dh, c.got_dw
    c.backward(lse, c.dloss, dweights=None)
    assert torch.equal(c.got_dh, dh)
    c.backward(lse, c.dloss, dhidden=None, dweights=[None, torch.empty_like(dw[1]), None])
    assert torch.equal(c.got_dw[1], dw[1])
    c.backward(lse, c.dloss, dhidden=c.hidden)
    assert torch.equal(c.hidden, dh) and all(torch.equal(a, b) for a, b in zip(c.got_dw, dw))


def test_backward_of_no_tokens_is_zero():
    announce("xent no tokens")
    for t in ("bf16", "f32"):
        w = torch.randn(9, 33, device="cuda").to(TYPES[t])
        d = torch.full_like(w, 3.0)
        mrr.check(mrr.mrr_linear_xent_bwd(None, [w], [9], 1, None, IGNORE, None, None, 1, None, [d], 0, 33, 33, 33, t))
        assert not bool(d.any())


@pytest.mark.parametrize("tokens", [7, 90, 300])
def test_gradients_are_the_slope_of_the_forward(tokens):
    """Along a direction of hidden states and weights: the gradients' slope against
    (L(e) - L(-e)) / 2e, L = <dloss, loss> in 64 bits from the f32 kernel's losses.
    Each loss is off by less than its tolerance; the step's own error falls with
    e^2, so that of e is a third of the difference between the slopes at e and 2e."""
    announce("xent slope", tokens)
    c = Case(tokens, [310, 200], 96, "f32", 13)
    c.forward()
    c.backward(c.got_lse.clone(), c.dloss)
    g = seeded(14)
    dirs = [torch.randn(x.shape, generator=g, device="cuda") * x.std() for x in [c.hidden] + c.weights]
    slope = sum(float((a.double() * b.double()).sum()) for a, b in zip([c.got_dh] + c.got_dw, dirs))
    at = [x.clone() for x in [c.hidden] + c.weights]

    def loss(e):
        for x, x0, d in zip([c.hidden] + c.weights, at, dirs):
            x.copy_(x0 + e * d)
        c.forward()
        c.exact()
        return float((c.dloss.double() * c.got_loss.double()).sum()), float((c.dloss.double() * c.eloss).sum())

    def measured(e):
        (p, ep), (m, em) = loss(e), loss(-e)
        # the points are rounded: u of each operand on the way, which the slopes carry over
        moved = sum(float((x.abs().double() * gr.abs().double()).sum()) for x, gr in zip(at, [c.got_dh] + c.got_dw))
        return (p - m) / (2 * e), (ep + em + 4 * U * moved) / (2 * e)

    (one, tol), (two, _) = measured(2.0 ** -7), measured(2.0 ** -6)
    assert abs(one - slope) <= abs(two - one) + tol + 1e-6 * abs(slope), (one, two, slope, tol)


@pytest.mark.parametrize("tokens", [3, 60, 400])
def test_another_stream_and_replays_of_a_graph(tokens):
    announce("xent graph", tokens)
    c = Case(tokens, [700, 300], 256, "bf16", 15)
    wf, wb = c.workspace(False), c.workspace(True)
    loss, lse = torch.empty(tokens, device="cuda"), torch.empty(tokens, device="cuda")
    dh, dw = torch.empty_like(c.hidden), [torch.empty_like(w) for w in c.weights]
    outs = [loss, lse, dh] + dw

    def step(stream=None):
        c.forward(loss=loss, lse=lse, stream=stream, ws=wf)
        c.backward(lse, c.dloss, dhidden=dh, dweights=dw, stream=stream, ws=wb)

    def eager(stream=None):
        step(stream)
        return [o.clone() for o in outs]

    want = eager()
    assert all(torch.equal(a, b) for a, b in zip(want, eager()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = eager(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(4):
        g = seeded(20 + k)
        c.hidden.copy_(torch.randn(c.hidden.shape, generator=g, device="cuda"))
        c.targets.copy_(torch.randint(0, 1000, (tokens,), generator=g, device="cuda"))
        c.targets[torch.rand(tokens, generator=g, device="cuda") < 0.1 * k] = IGNORE
        want = eager()
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, outs)), k


@pytest.mark.parametrize("tokens", [2, 50, 300])
@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_the_small_loss_of_a_sure_token_keeps_its_digits(tokens, t):
    """A target's logit of 25 above all others, which are 0 (rows of zeros): the loss is
    log(1 + (V - 1) exp(-25)), and only its sum's rounding (2 u of 1, twice for the pieces
    it is joined from) and log's are between.  lse is off by its own rounding as well."""
    announce("xent sure", tokens, t)
    vocab, cols = 3000, 64
    w = torch.zeros(vocab, cols, dtype=TYPES[t], device="cuda")
    w[1234, 0] = 5.0
    h = torch.zeros(tokens, cols, dtype=TYPES[t], device="cuda")
    h[:, 0] = 5.0
    targets = torch.full((tokens,), 1234, dtype=torch.int64, device="cuda")
    loss, lse = torch.empty(tokens, device="cuda"), torch.empty(tokens, device="cuda")
    n = mrr.mrr_linear_xent_workspace_bytes(tokens, cols, [1000, 2000], 2, t, False)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    mrr.check(mrr.mrr_linear_xent_fwd(h, [w[:1000], w[1000:]], [1000, 2000], 2, targets, IGNORE, loss, lse, tokens, cols, cols,
                                      cols, t, ws, n))
    want = float(torch.log1p(2999 * torch.exp(torch.tensor(-25.0, dtype=torch.float64))))
    assert float((loss.double() - want).abs().max()) <= 4 * U + 2 * U * want
    assert float((lse.double() - 25 - want).abs().max()) <= 4 * U + U * 26


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("tokens", [3, 6])
def test_rows_four_gigabytes_apart(tokens, t):
    """Operands and gradients are columns of one buffer whose rows are 2^31 elements apart."""
    announce("xent far rows", tokens, t)
    c = Case(tokens, [5], 72, t, 40)
    ld = 1 << 31
    room = torch.empty(5 * ld + 1024, dtype=TYPES[t], device="cuda")
    view = [room.as_strided((n, 72), (ld, 1), 128 * k) for k, n in enumerate((tokens, 5, tokens, 5))]
    view[0].copy_(c.hidden)
    view[1].copy_(c.weights[0])
    c.hidden, c.weights, c.ld = view[0], [view[1]], ld
    c.forward()
    torch.cuda.synchronize()
    c.check_forward()
    lse = c.lse.float()
    c.backward(lse, c.dloss, dhidden=view[2], dweights=[view[3]])
    torch.cuda.synchronize()
    c.exact(lse, c.dloss)
    c.check_backward()


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("tokens,rows,cols", [(5, [700, 3], 192), (17, [512, 300], 640), (40, [100] * 4, 1024), (64, [260], 128),
                                              (64, [4000], 64), (100, [900, 40], 72), (300, [1000], 65), (1000, [130], 64)])
def test_both_sides_of_the_rule_for_few_tokens(tokens, rows, cols, t):
    """The shapes at which the way to the logits changes, hidden states in place and not."""
    announce("xent few", t, tokens, rows, cols)
    for pad in (0, 8, 1):
        c = Case(tokens, rows, cols, t, tokens + cols + pad, pad=pad)
        c.forward()
        torch.cuda.synchronize()
        c.check_forward()
        lse = c.lse.float()
        c.backward(lse, c.dloss)
        torch.cuda.synchronize()
        c.exact(lse, c.dloss)
        c.check_backward()
