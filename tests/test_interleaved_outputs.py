"""CPU checks of outputs that lie between each other in one buffer without sharing a byte: heads of the queries, keys and
values in turn, column slices of a batch of matrices.  Pointers are fake device addresses that no call here reaches."""
import random

import pytest
import torch

import allreduce_reduction_nranks_amd as mrr

BASE = 0x7F0000000000
E = 2  # bytes of an element


def fake(i, elements=0):
    return BASE + (i << 34) + E * elements


def fwd(tokens, heads, dim, places, lds, strides, inputs=None, ld_in=None):
    """The status of a forward whose outputs lie `places` elements into one buffer (None: not wanted)."""
    outs = [None if p is None else fake(9, p) for p in places]
    return mrr.STATUS_NAMES[mrr.mrr_qknorm_rope_fwd(inputs or [fake(0)], 1, None, None, None, 0, None, None, outs, tokens, heads, dim, 0, False,
                                                    ld_in or sum(heads) * dim, lds, strides, 1e-6, "bf16", stream=0)]


def no_gpu():
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real")


@pytest.mark.parametrize("tokens", [1, 2, 16])
@pytest.mark.parametrize("pad", [0, 5])
@pytest.mark.parametrize("n,dim", [(4, 64), (3, 41), (1, 16)])
def test_heads_of_queries_keys_and_values_in_turn(tokens, pad, n, dim):
    no_gpu()
    ld = 3 * n * dim + pad
    assert fwd(tokens, [n] * 3, dim, [0, dim, 2 * dim], [ld] * 3, [3 * dim] * 3) == "MRR_EHIP"
    assert fwd(tokens, [n] * 3, dim, [2 * dim, 0, dim], [ld] * 3, [3 * dim] * 3) == "MRR_EHIP"
    # each head's tokens side by side, of the queries, keys and values in turn
    ld = 3 * dim + pad
    assert fwd(tokens, [n] * 3, dim, [0, dim, 2 * dim], [ld] * 3, [ld * tokens] * 3) == "MRR_EHIP"
    # two key and value heads beside the queries', which lie apart
    assert fwd(tokens, [n, 2, 2], dim, [4 * dim, 0, dim], [(n + 4) * dim] * 3, [dim, 2 * dim, 2 * dim]) == "MRR_EHIP"


@pytest.mark.parametrize("tokens", [1, 2, 16])
def test_one_element_too_near(tokens):
    n, dim = 4, 64
    for places in ([0, dim - 1, 2 * dim], [0, dim, 3 * dim - 1], [0, dim, 3 * dim + 1], [0, 0, dim], [dim, 2 * dim - 1, 0]):
        ld = 3 * n * dim + 70
        assert fwd(tokens, [n] * 3, dim, places, [ld] * 3, [3 * dim] * 3) == "MRR_EOVERLAP", places
    # the last head of one token and the first of the next
    assert fwd(2, [n] * 3, dim, [0, dim, 2 * dim + 1], [3 * n * dim] * 3, [3 * dim] * 3) == "MRR_EOVERLAP"


def touched(tokens, heads, dim, place, ld, stride):
    return {place + t * ld + j * stride + d for t in range(tokens) for j in range(heads) for d in range(dim)}


def test_random_layouts_that_share_an_element_are_refused():
    no_gpu()
    rng = random.Random(3)
    seen = {"MRR_EHIP": 0, "MRR_EOVERLAP": 0}
    for _ in range(4000):
        tokens, n, dim = rng.randint(1, 4), [rng.randint(1, 4), rng.randint(1, 4)], rng.randint(1, 6)
        stride = rng.randint(dim, 4 * dim)
        ld = stride * max(n) + rng.randint(0, 6)
        lds, strides = [ld, ld], [stride, stride]
        if rng.random() < 0.3:
            strides[1] = rng.randint(dim, 4 * dim)
            lds[1] = max(ld, strides[1] * n[1])
        if rng.random() < 0.3:
            lds, strides = [s for s in strides], [max(strides) * tokens + rng.randint(0, 5)] * 2
        places = [rng.randint(0, 2 * ld), rng.randint(0, 2 * ld)]
        got = fwd(tokens, n + [0], dim, places + [None], lds + [0], strides + [0])
        shared = bool(touched(tokens, n[0], dim, places[0], lds[0], strides[0]) & touched(tokens, n[1], dim, places[1], lds[1], strides[1]))
        assert got == "MRR_EOVERLAP" or (got == "MRR_EHIP" and not shared), (tokens, n, dim, places, lds, strides)
        seen[got] += 1
    assert min(seen.values()) > 500


def muon(places, ld, batch=3, rows=40, cols=50, stride=None):
    """weight, momentum, momentum_out and the new weights of two ranks, f32, `places` elements into one buffer."""
    w, m, mo, w0, w1 = [fake(9, 2 * p) for p in places]
    n = mrr.mrr_muon_workspace_bytes(rows, cols, batch, "f32")
    return mrr.STATUS_NAMES[mrr.mrr_muon_step([fake(0), fake(1)], 2, 0.5, m, mo, 0.9, True, w, [w0, w1], 0.02, 0.0, rows, cols, cols, ld, batch,
                                              rows * cols, rows * ld if stride is None else stride, 5, None, 1e-7, "f32", "f32",
                                              workspace=fake(5), workspace_bytes=n, stream=0)]


def test_column_slices_of_a_batch_of_matrices():
    no_gpu()
    cols = 50
    for ld in (5 * cols, 5 * cols + 7):
        assert muon([k * cols for k in range(5)], ld) == muon([k * cols for k in (3, 1, 4, 0, 2)], ld) == "MRR_EHIP"
        assert muon([0, cols, cols, 2 * cols, 3 * cols], ld) == muon([0, cols, 2 * cols, 0, 3 * cols], ld) == "MRR_EHIP"
        assert muon([k * cols for k in range(5)], ld, stride=50 * ld) == "MRR_EHIP"
        for k in range(2, 5):  # (the first two are read, and may overlap)
            places = [j * cols for j in range(5)]
            places[k] -= 1
            assert muon(places, ld) == "MRR_EOVERLAP", k
