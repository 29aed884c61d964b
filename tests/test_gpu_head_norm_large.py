"""GPU checks of the head norms' kernels for calls that move more than the caches hold, which smaller calls do not reach, against
the formulas in 64 bits with test_gpu_qknorm's tolerances: waves that walk over tokens, one rank; several ranks past the caches;
the gradient past them.  And of more tokens than a grid has waves.  Each case says which kernel it is for."""
import pytest
import torch

import allreduce_reduction_nranks_amd as mrr
from gpu_common import announce
from kernels_run import kernels_of, template_of
from test_gpu_qknorm import ROWS, TYPES, backward, check_forward, empty_outs, forward, randn, seeded, table_of

pytestmark = pytest.mark.gpu

CACHE = 256 << 20
CODES = {"f32": "1", "f16": "2", "bf16": "3"}  # a type as a kernel's template argument

# type, heads, elements of a head, rotated, neighbours in pairs, lanes of a head: heads with nothing to mask of every lane
# count, and masked ones that do not fill a wave, end inside a vector or rotate in part
SHAPES = [("bf16", (32, 8, 8), 128, 128, False, 8), ("f16", (3, 1, 2), 64, 64, True, 4), ("bf16", (2, 1, 1), 256, 256, True, 16),
          ("f16", (2, 2, 1), 512, 512, False, 32), ("f32", (4, 2, 2), 32, 32, False, 4), ("f32", (12, 12, 12), 64, 64, True, 8),
          ("f32", (3, 1, 1), 128, 128, False, 16), ("f32", (1, 1, 1), 256, 256, True, 32), ("f32", (2, 1, 0), 512, 512, False, 64),
          ("f16", (5, 3, 1), 80, 32, True, 8), ("f16", (7, 1, 1), 96, 48, False, 8), ("bf16", (32, 8, 8), 128, 64, False, 8),
          ("f32", (6, 2, 2), 112, 56, False, 16), ("bf16", (1, 1, 1), 20, 20, True, 4), ("bf16", (9, 3, 0), 68, 0, False, 8),
          ("f32", (3, 2, 1), 53, 26, True, 8), ("f32", (1, 0, 2), 300, 100, True, 64)]


def tokens_of(t, heads, dim, moves):
    """Some more tokens than move CACHE bytes; moves: of a token, in heads."""
    return int(CACHE * 1.02) // (moves * dim * torch.finfo(TYPES[t]).bits // 8) + 3


def positions_of(g, tokens):
    """Runs of padded tokens, the first and the last among them."""
    p = torch.randint(0, ROWS, (tokens,), generator=g, device="cuda")
    at = torch.arange(tokens, device="cuda")
    p[(at % 1001 < 37) | (at % 7 == 3)] = -1
    p[-5:] = -2
    return p


def untouched(tensors, positions):
    return all(bool((x[positions < 0] == 7.0).all()) for x in tensors if x is not None)


def main_kernel(call):
    return template_of(kernels_of(call)[0])


@pytest.mark.parametrize("t,heads,dim,rot,pairs,lanes", SHAPES)
@pytest.mark.parametrize("unit_weight", [False, True])
def test_one_rank(t, heads, dim, rot, pairs, lanes, unit_weight):
    announce("qk walk", t, heads, dim, rot, pairs, unit_weight)
    tokens = tokens_of(t, heads, dim, 2 * sum(heads))
    g = seeded(dim + rot)
    x = randn(g, tokens, sum(heads) * dim, t=t, shift=0.1)
    tw = "f32" if dim % 3 else t
    weights = [randn(g, dim, t=tw, shift=1.0), None if unit_weight else randn(g, dim, t=tw, shift=1.0)]
    positions, table, outs = positions_of(g, tokens), table_of(rot), empty_outs(tokens, heads, dim, t)
    name, args = main_kernel(lambda: mrr.check(forward([x], weights, table, positions, None, outs, list(heads), dim, rot, pairs, t, tw)))
    assert name == "qk_walk_k" and args == [CODES[t], str(16 // (4 if t == "f32" else 2)), str(lanes), str(pairs).lower(),
                                            str(rot == dim and dim * (4 if t == "f32" else 2) == 32 * lanes).lower()]
    check_forward([x], weights, table, positions, None, outs, heads, dim, rot, pairs, t)
    assert untouched(outs, positions)


@pytest.mark.parametrize("dim,rot,pairs", [(128, 128, False), (80, 32, True)])
def test_one_rank_in_place_with_a_sum_and_an_output_not_wanted(dim, rot, pairs):
    announce("qk walk in place", dim)
    heads, t = [5, 3, 2], "bf16"
    tokens = tokens_of(t, heads, dim, 2 * 10)
    g = seeded(dim)
    x = randn(g, tokens, 10 * dim, t=t)
    weights, positions, table = [None, randn(g, dim)], positions_of(g, tokens), table_of(rot)
    want = empty_outs(tokens, heads, dim, t)
    mrr.check(forward([x], weights, table, positions, None, want, heads, dim, rot, pairs, t, "f32"))
    total, one = torch.full_like(x, 7.0), empty_outs(tokens, heads, dim, t)
    run = lambda: mrr.check(forward([x], weights, table, positions, total, [None] + one[1:], heads, dim, rot, pairs, t, "f32"))  # noqa: E731
    assert main_kernel(run)[0] == "qk_walk_k"
    live = positions >= 0
    assert all(torch.equal(a, b) for a, b in zip(one[1:], want[1:])) and torch.equal(total[live], x[live]) and untouched([total], positions)
    y = x.clone()
    places = list(y.split([n * dim for n in heads], 1))
    run = lambda: mrr.check(forward([y], weights, table, positions, None, places, heads, dim, rot, pairs, t, "f32", lds=[10 * dim] * 3))  # noqa: E731
    assert main_kernel(run)[0] == "qk_walk_k"
    assert torch.equal(y[live], torch.cat([o.flatten(1) for o in want], 1)[live]) and torch.equal(y[~live], x[~live])


@pytest.mark.parametrize("t,heads,dim,rot,pairs,lanes", [SHAPES[k] for k in (0, 1, 5, 8, 9, 10, 12, 16)])
@pytest.mark.parametrize("ranks,group", [(2, 2), (3, 4), (4, 4), (5, 8), (8, 8), (11, 8)])
def test_several_ranks(t, heads, dim, rot, pairs, lanes, ranks, group):
    announce("qk ranks past the caches", t, heads, dim, rot, pairs, ranks)
    tokens = tokens_of(t, heads, dim, (ranks + 2) * sum(heads))
    g = seeded(dim + ranks)
    inputs = [randn(g, tokens, sum(heads) * dim, t=t, shift=0.1) for _ in range(ranks)]
    weights = [randn(g, dim, shift=1.0), randn(g, dim, shift=1.0)]
    positions, table, outs = positions_of(g, tokens), table_of(rot), empty_outs(tokens, heads, dim, t)
    total = torch.full_like(inputs[0], 7.0)
    run = lambda: mrr.check(forward(inputs, weights, table, positions, total, outs, list(heads), dim, rot, pairs, t, "f32"))  # noqa: E731
    name, args = main_kernel(run)
    assert name == "qk_fwd_k" and args[2] == str(lanes) and args[4] == str(group) and args[-1] == "true"
    check_forward(inputs, weights, table, positions, total, outs, heads, dim, rot, pairs, t)
    assert untouched(outs + [total], positions)
    # the sum in an input's place
    want = total.clone()
    want[positions < 0] = inputs[-1][positions < 0]
    mrr.check(forward(inputs, weights, table, positions, inputs[-1], [None] * 3, list(heads), dim, rot, pairs, t, "f32"))
    assert torch.equal(inputs[-1], want)


@pytest.mark.parametrize("t,heads,dim,rot,pairs,lanes", SHAPES)
def test_gradient(t, heads, dim, rot, pairs, lanes):
    announce("qk gradient past the caches", t, heads, dim, rot, pairs)
    tokens = tokens_of(t, heads, dim, 3 * sum(heads) - heads[2])
    g = seeded(dim + rot)
    h = randn(g, tokens, sum(heads) * dim, t=t, shift=0.1)
    weights = [randn(g, dim, shift=1.0), randn(g, dim, shift=1.0)]
    positions, table = positions_of(g, tokens), table_of(rot)
    douts = [randn(g, tokens, n, dim, t=t) if n else None for n in heads]
    h[positions < 0] = float("nan")  # not read
    for d in douts:
        if d is not None:
            d[positions < 0] = float("inf")
    dsum, dws = torch.full_like(h, 7.0), [torch.full((dim,), 7.0, device="cuda") for _ in range(2)]
    run = lambda: mrr.check(backward(douts, h, weights, table, positions, dsum, dws, list(heads), dim, rot, pairs, t, "f32"))  # noqa: E731
    name, args = main_kernel(run)
    assert name == "qk_bwd_k" and args[2] == str(lanes) and args[-1] == "true"
    check_large_backward(douts, h, weights, table, positions, dsum, dws, heads, dim, rot, pairs, t)
    assert not bool(dsum[positions < 0].any())
    again, dws2 = h.clone(), [torch.full_like(d, 7.0) for d in dws]
    mrr.check(backward(douts, again, weights, table, positions, again, dws2, list(heads), dim, rot, pairs, t, "f32"))
    assert torch.equal(again, dsum) and all(torch.equal(a, b) for a, b in zip(dws2, dws))


def check_large_backward(douts, h, weights, table, positions, dsum, dws, heads, dim, rot, pairs, t):
    """check_backward, whose 256 steps of a weight's sum are for up to 128 terms of a lane: here as many of the tokens as fall to one
    of 768 * 4 waves, each of heads / (64 / lanes) iterations at most, follow each other in a lane.  Its tolerance holds for
    as many more."""
    import test_gpu_qknorm as q
    terms = (len(h) / (768 * 4) + 1) * (max(heads) + 1)
    want, tol, dw, tdw = q.backward_tolerances(douts, h, weights, table, positions, heads, dim, rot, pairs, t)
    q.close(dsum, want, tol, "dsum")
    for k in range(2):
        q.close(dws[k], dw[k], q.U * dw[k].abs() + tdw[k] * max(1.0, (terms + 128) / 256) * (1 + q.U), "d%s_weight" % "qk"[k])


@pytest.mark.parametrize("ranks", [1, 2])
def test_more_tokens_than_a_grid_has_waves(ranks):
    announce("qk token stride", ranks)
    heads, dim, t = [1, 1, 1], 2, "f32"
    tokens = (1 << 24) // 3 + 12345
    g = seeded(ranks)
    inputs = [randn(g, tokens, 6) for _ in range(ranks)]
    weights, positions, table = [randn(g, dim), randn(g, dim)], positions_of(g, tokens), table_of(2)
    total, outs = torch.full_like(inputs[0], 7.0), empty_outs(tokens, heads, dim, t)
    run = lambda: mrr.check(forward(inputs, weights, table, positions, total, outs, heads, dim, 2, False, t, t))  # noqa: E731
    assert main_kernel(run)[0] == "qk_fwd_k"
    check_forward(inputs, weights, table, positions, total, outs, heads, dim, 2, False, t)
    assert untouched(outs + [total], positions)
