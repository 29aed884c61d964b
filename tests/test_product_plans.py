"""CPU checks that the shapes which tests take for a way of the products are still planned that way: a change of the planner's
times that sends one elsewhere fails here, not silently there."""
import random

import pytest

import allreduce_reduction_nranks_amd as mrr
from product_plans import SHAPES, plan, ways


@pytest.mark.parametrize("sides,batch,parts,gram,square,apply", SHAPES)
def test_each_shape_has_its_ways(sides, batch, parts, gram, square, apply):
    assert ways(*sides, batch, parts) == ways(*sides[::-1], batch, parts) == (gram, square, apply)


def test_the_plan_is_the_call_s():
    """What is read here is what the entry points use: its last field is the workspace's size."""
    for sides, batch, parts, *_ in SHAPES:
        p = plan(*sides, batch, parts)
        assert p.parts == parts and p.bytes == mrr.mrr_orthogonalize_workspace_bytes(*sides, batch, "bf16", "f16" if parts == 1 else "f32")


def test_no_shape_has_another_way():
    rng = random.Random(12)
    known = {(s[2], k, s[3 + k]) for s in SHAPES for k in range(3)}
    for _ in range(20000):
        a, b = (int(2 ** rng.uniform(0, 16)) for _ in range(2))
        if rng.random() < 0.5:
            a, b = ((x + 63) // 64 * 64 for x in (a, b))
        batch = 1 if rng.random() < 0.4 else int(2 ** rng.uniform(0, min(16, 34 - (a * b).bit_length()) - 0.01))
        for parts in (1, 2):
            if parts == 2 or min(a, b) > 64:
                new = {(parts, k, w) for k, w in enumerate(ways(a, b, max(1, batch), parts))} - known
                assert not new, (a, b, batch, new)
