"""CPU check that the tolerances of tests/xent_few_tokens.py see a dz held in one 16-bit part, with
and without its targets' residue."""
import pytest
import torch

from xent_few_tokens import TYPES, Few


def gradients(c, parts, residue):
    scale = 2.0 ** 13 if c.t == "f16" else 1.0
    held, left = torch.zeros_like(c.dz), c.dz * scale
    for _ in range(parts):
        part = left.to(TYPES[c.t]).double()
        held, left = held + part, left - part
    dz = (held + (c.hit * left if residue else 0.0)) / scale
    return (dz @ c.w).to(TYPES[c.t]), (dz.T.contiguous() @ c.h).to(TYPES[c.t])


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("tokens", [1, 4, 64])
def test_one_part_is_seen(tokens, t):
    c = Few(tokens, [300, 600], 128, t, 1, "cpu")
    assert c.off(*gradients(c, 2, False)) == [0, 0]
    for residue in (False, True):
        assert c.off(*gradients(c, 1, residue))[1] > 0
