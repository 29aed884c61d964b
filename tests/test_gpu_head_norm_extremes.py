"""GPU checks of mrr_qknorm_rope_fwd and _bwd where a call is unusual: places past 32 bits, the most heads, one rank's
pointer several times, calls on two streams at once, two graphs with one workspace.  A result must be bit for bit that of
the ordinary call."""
import pytest
import torch

import allreduce_reduction_nranks_amd as mrr
from gpu_common import announce
from test_gpu_qknorm import TYPES, backward, check_forward, empty_outs, forward, randn, seeded, table_of

pytestmark = pytest.mark.gpu


def far(n):
    """n bf16 elements, none of them written."""
    return torch.empty(n, dtype=torch.bfloat16, device="cuda")


@pytest.mark.parametrize("dim,rot", [(64, 64), (41, 20)])
@pytest.mark.parametrize("way", ["heads", "tokens", "rows"])
def test_places_past_32_bits(way, dim, rot):
    announce("qk far", way, dim, rot)
    g = seeded(31)
    tokens, heads = 3, [3, 1, 1]
    width = sum(heads) * dim
    table, weights = table_of(rot), [randn(g, dim), randn(g, dim)]
    inputs = [randn(g, tokens, width, t="bf16") for _ in range(2)]
    want, total, dsum = empty_outs(tokens, heads, dim, "bf16"), torch.empty_like(inputs[0]), torch.empty_like(inputs[0])
    dws = [torch.empty(dim, device="cuda") for _ in range(2)]
    mrr.check(forward(inputs, weights, table, None, total, want, heads, dim, rot, False, "bf16", "f32"))
    douts = [randn(g, tokens, n, dim, t="bf16") for n in heads]
    mrr.check(backward(douts, total, weights, table, None, dsum, dws, heads, dim, rot, False, "bf16", "f32"))

    side = 1 << 31
    ld, strides, ld_in = [n * dim for n in heads], [dim] * 3, width
    if way == "heads":     # queries: heads past 2^31 elements from each other
        ld[0], strides[0] = dim, side + 5
        size = 2 * strides[0] + tokens * dim
    elif way == "tokens":  # tokens as far apart as may be
        ld[0] = side
        size = 2 * side + heads[0] * dim
    if way == "rows":      # of the inputs, the sum and its gradient
        buffers = [far(2 * side + width) for _ in range(2)]
        rows = [b.as_strided((tokens, width), (side, 1)) for b in buffers]
        for to, x in zip(rows, inputs):
            to.copy_(x)
        outs = empty_outs(tokens, heads, dim, "bf16")
        mrr.check(forward(rows, weights, table, None, rows[0], outs, heads, dim, rot, False, "bf16", "f32", ld_in=side))
        assert torch.equal(rows[0], total)
        got_dws = [torch.empty_like(w) for w in dws]
        mrr.check(backward(douts, rows[0], weights, table, None, rows[1], got_dws, heads, dim, rot, False, "bf16", "f32", ld_in=side))
        assert torch.equal(rows[1], dsum)
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    else:
        buffer = far(size)
        view = buffer.as_strided((tokens, heads[0], dim), (ld[0], strides[0], 1))
        outs = [view] + empty_outs(tokens, heads, dim, "bf16")[1:]
        mrr.check(forward(inputs, weights, table, None, None, outs, heads, dim, rot, False, "bf16", "f32", lds=ld, strides=strides))
        assert torch.equal(view, want[0]) and torch.equal(outs[1], want[1])
        view.copy_(douts[0])
        got, got_dws = torch.empty_like(dsum), [torch.empty_like(w) for w in dws]
        mrr.check(backward([view] + douts[1:], total, weights, table, None, got, got_dws, heads, dim, rot, False, "bf16", "f32", lds=ld,
                           strides=strides))
        assert torch.equal(got, dsum)
    assert all(torch.equal(a, b) for a, b in zip(got_dws, dws))


@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_the_most_heads(t):
    announce("qk most heads", t)
    g = seeded(32)
    tokens, heads, dim = 2, [65535, 65535, 65535], 16
    x = randn(g, tokens, sum(heads) * dim, t=t)
    weights = [randn(g, dim, t=t), None]
    outs = empty_outs(tokens, heads, dim, t)
    table = table_of(dim)
    mrr.check(forward([x], weights, table, None, None, outs, heads, dim, dim, True, t, t))
    check_forward([x], weights, table, torch.arange(tokens, device="cuda"), None, outs, heads, dim, dim, True, t)


def test_one_rank_several_times():
    announce("qk one rank several times")
    g = seeded(33)
    tokens, heads, dim = 130, [2, 1, 1], 64
    x = randn(g, tokens, 4 * dim, t="f16")
    weights, table = [randn(g, dim), randn(g, dim)], table_of(dim)
    want, got = (empty_outs(tokens, heads, dim, "f16") for _ in range(2))
    total, sums = torch.empty_like(x), x.clone()
    mrr.check(forward([x.clone(), x.clone(), x.clone()], weights, table, None, total, want, heads, dim, dim, False, "f16", "f32"))
    mrr.check(forward([sums, sums, sums], weights, table, None, sums, got, heads, dim, dim, False, "f16", "f32"))
    assert torch.equal(sums, total) and all(torch.equal(a, b) for a, b in zip(got, want))


def call(seed, t, tokens=700):
    """A forward and backward with buffers of its own."""
    g = seeded(seed)
    heads, dim, rot = [6, 2, 2], 128, 128
    inputs = [randn(g, tokens, 10 * dim, t=t) for _ in range(3)]
    table, weights = table_of(rot, 1024), [randn(g, dim), randn(g, dim)]
    douts = [randn(g, tokens, n, dim, t=t) for n in heads]
    outs, total, dsum = empty_outs(tokens, heads, dim, t), torch.empty_like(inputs[0]), torch.empty_like(inputs[0])
    dws = [torch.empty(dim, device="cuda") for _ in range(2)]
    n = mrr.mrr_qknorm_rope_bwd_workspace_bytes(tokens, heads, dim)
    own = torch.empty(n, dtype=torch.uint8, device="cuda")

    def run(ws=own):
        mrr.check(forward(inputs, weights, table, None, total, outs, heads, dim, rot, False, t, "f32"))
        mrr.check(backward(douts, total, weights, table, None, dsum, dws, heads, dim, rot, False, t, "f32", ws=ws))
    return run, outs + [total, dsum] + dws


def test_two_streams_at_once():
    announce("qk two streams")
    calls = [call(34, "bf16"), call(35, "f32")]
    want = []
    for run, results in calls:
        run()
        torch.cuda.synchronize()
        want.append([r.clone() for r in results])
        for r in results:
            r.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(20):
        for s, (run, _) in zip(streams, calls):
            with torch.cuda.stream(s):
                run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for (_, results), w in zip(calls, want) for a, b in zip(results, w))


def test_two_graphs_with_one_workspace():
    announce("qk two graphs")
    calls = [call(36, "bf16", 90), call(37, "bf16", 1000)]
    ws = torch.empty(mrr.mrr_qknorm_rope_bwd_workspace_bytes(1000, [6, 2, 2], 128), dtype=torch.uint8, device="cuda")
    want, graphs = [], []
    for run, results in calls:
        run(ws)
        torch.cuda.synchronize()
        want.append([r.clone() for r in results])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run(ws)
        graphs.append(graph)
    for _ in range(3):
        for _, results in calls:
            for r in results:
                r.zero_()
        ws.fill_(255)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for (_, results), w in zip(calls, want) for a, b in zip(results, w))
