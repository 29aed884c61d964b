"""Coefficients whose largest singular value lies inside the range of the ones before, on the CPU: a call is refused where one
before a later step could come within 1 % of 7.5, wherever the polynomial has its maximum."""
import random

import pytest
import torch

import allreduce_reduction_nranks_amd as mrr

BASE = 0x7F0000000000


def orth(co):
    steps = len(co) // 3
    n = mrr.mrr_orthogonalize_workspace_bytes(96, 160, 1, "f32")
    return mrr.STATUS_NAMES[mrr.mrr_orthogonalize(BASE, BASE + (1 << 34), 96, 160, 160, 160, 1, 0, 0, steps, co, 1e-7, "f32", "auto",
                                                  BASE + (2 << 34), n, stream=0)]


# 6 s - 0.4 s^3 has its maximum, 8.94, at s = 2.24, and is -1.6 at 4.04, where the range of the step before ends
@pytest.mark.parametrize("c", [0.0] + [s * 10.0 ** -k for k in (6, 12, 17, 18, 20, 30, 38, 45) for s in (1, -1)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_a_maximum_inside_is_seen_beside_a_tiny_coefficient(c, sign):
    assert orth((4.0, 0.0, 0.0, sign * 6.0, sign * -0.4, sign * c, 1.0, 0.0, 0.0)) == "MRR_EINVAL"


def largest(co):
    """The largest singular value before the last step and the largest |b x + c x^2|, of 4001 values each, 1 % above each step's."""
    top, most, before = 1.0, 0.0, 0.0
    for k in range(0, len(co), 3):
        a, b, c = co[k:k + 3]
        before = max(before, top)
        s = torch.linspace(0.0, top, 4001, dtype=torch.float64)
        x = s * s
        most = max(most, float((b * x + c * x * x).abs().max()))
        top = 1.01 * float((s * (a + b * x + c * x * x)).abs().max())
    return before, most


def test_random_coefficients():
    """Against the largest of many values; a parabola's between two of 4001 points are at most 1e-4 above them, so that what lies
    within 1e-3 of a limit is left out."""
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real")
    rng = random.Random(7)
    seen = {True: 0, False: 0}
    for _ in range(3000):
        co = []
        for _ in range(rng.choice([2, 3])):
            b = rng.choice([-1, 1]) * 10.0 ** rng.uniform(-3, 1)
            c = rng.choice([0.0, rng.choice([-1, 1]) * 10.0 ** rng.choice([rng.uniform(-3, 1), rng.uniform(-45, -6)])])
            co += [rng.uniform(-6, 6), b, c]
        co = torch.tensor(co, dtype=torch.float32).tolist()
        before, most = largest(co)
        if abs(before / 7.5 - 1) < 1e-3 or abs(most / 1000 - 1) < 1e-3:
            continue
        refused = before >= 7.5 or most >= 1000
        assert orth(co) == ("MRR_EINVAL" if refused else "MRR_EHIP"), co
        seen[refused] += 1
    assert min(seen.values()) > 300
