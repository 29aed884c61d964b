"""CPU check that the tolerances of tests/xent_residue.py see what they are for: gradients from a dz
rounded to 16 bits are outside them without its targets' residue, with it twice, or with
another token's."""
import pytest
import torch

from xent_residue import TYPES, Targets


def gradients(c, residue):
    scale = 2.0 ** 13 if c.t == "f16" else 1.0
    held = (c.dz * scale).to(TYPES[c.t]).double() / scale
    lost = torch.where(c.hit > 0, c.dz - held, 0.0).sum(1)
    dz = held + c.hit * residue(lost)[:, None]
    return (dz @ c.w).to(TYPES[c.t]), (dz.T.contiguous() @ c.h).to(TYPES[c.t])


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("tokens,rows,cols", [(30, [600, 300], 128), (200, [600, 300], 128)])
def test_a_wrong_residue_is_seen(tokens, rows, cols, t):
    c = Targets(tokens, rows, cols, t, 1, "cpu")
    assert c.share_off(*gradients(c, lambda lost: lost)) == [0.0, 0.0]
    for wrong in (lambda lost: 0 * lost, lambda lost: 2 * lost, lambda lost: lost.roll(1)):
        assert min(c.share_off(*gradients(c, wrong))) > 0.0
