"""GPU checks of when the head norms go past the caches: by what a call moves, not by how far its rows lie apart or by a part of a
long row.  The rule: more than 256 MiB of elements read and written."""
import pytest
import torch

import allreduce_reduction_nranks_amd as mrr
from gpu_common import announce
from kernels_run import kernels_of, template_of
from test_gpu_qknorm import TYPES, backward, empty_outs, forward, randn, seeded, table_of

pytestmark = pytest.mark.gpu


def streams(call):
    """Whether the call's main kernel goes past the caches: the walk, or the last template argument of the others."""
    name, args = template_of(kernels_of(call)[0])
    assert name in ("qk_walk_k", "qk_fwd_k", "qk_bwd_k")
    return name == "qk_walk_k" or args[-1] == "true"


@pytest.mark.parametrize("ranks", [1, 2])
def test_columns_of_a_wide_buffer_count_as_what_they_are(ranks):
    announce("qk wide", ranks)
    g = seeded(ranks)
    tokens, heads, dim, ld = 3000, [1, 1, 1], 64, 65536
    wide = [torch.empty(tokens, ld, dtype=torch.bfloat16, device="cuda") for _ in range(ranks)]
    x = [w[:, 1000:1000 + 3 * dim] for w in wide]
    for v in x:
        v.copy_(randn(g, tokens, 3 * dim))
    outs, want = empty_outs(tokens, heads, dim, "bf16"), empty_outs(tokens, heads, dim, "bf16")
    table, weights = table_of(dim, tokens), [randn(g, dim), None]
    run = lambda: mrr.check(forward(x, weights, table, None, None, outs, heads, dim, dim, False, "bf16", "f32", ld_in=ld))  # noqa: E731
    assert not streams(run)
    mrr.check(forward([v.contiguous() for v in x], weights, table, None, None, want, heads, dim, dim, False, "bf16", "f32"))
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    dx, dws = wide[-1][:, 2000:2000 + 3 * dim], [torch.empty(dim, device="cuda") for _ in range(2)]
    assert not streams(lambda: mrr.check(backward(want, x[0], weights, table, None, dx, dws, heads, dim, dim, False, "bf16", "f32", ld_in=ld)))


@pytest.mark.parametrize("ranks", [1, 2])
def test_rows_of_very_many_heads_count_whole(ranks):
    announce("qk long rows", ranks)
    g = seeded(ranks)
    tokens, heads, dim = 160, [8000, 16, 16], 64
    width = sum(heads) * dim
    x = [randn(g, tokens, width, t="bf16") for _ in range(ranks)]
    outs = empty_outs(tokens, heads, dim, "bf16")
    table, weights = table_of(dim, tokens), [randn(g, dim), None]
    assert streams(lambda: mrr.check(forward(x, weights, table, None, None, outs, heads, dim, dim, False, "bf16", "f32")))
    dx, dws = torch.empty_like(x[0]), [torch.empty(dim, device="cuda") for _ in range(2)]
    assert streams(lambda: mrr.check(backward(outs, x[0], weights, table, None, dx, dws, heads, dim, dim, False, "bf16", "f32")))


@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_each_side_of_the_rule(t):
    """12 heads of 64: a token of one rank moves 12 * 64 * 2 elements forward, and 11 + 12 + 12 heads of them backward."""
    announce("qk rule", t)
    g = seeded(3)
    heads, dim = [8, 3, 1], 64
    size = torch.finfo(TYPES[t]).bits // 8
    table, weights = table_of(dim, 1 << 17), [None, None]
    for moved, run in ((24, "forward"), (35, "backward")):
        most = (256 << 20) // (moved * dim * size)
        for tokens, past in ((most, False), (most + 1, True)):
            x = torch.ones(tokens, 12 * dim, dtype=TYPES[t], device="cuda")
            outs = empty_outs(tokens, heads, dim, t)
            dx, dws = torch.empty_like(x), [torch.empty(dim, device="cuda") for _ in range(2)]
            if run == "forward":
                got = streams(lambda: mrr.check(forward([x], weights, table, None, None, outs, heads, dim, dim, False, t, "f32")))
            else:
                got = streams(lambda: mrr.check(backward(outs, x, weights, table, None, dx, dws, heads, dim, dim, False, t, "f32")))
            assert got == past, (run, tokens)
