"""GPU check of what cross entropy gradients in 16 bits give back of a target's dz: as a second
part of it (up to 64 tokens) and by tokens sorted by their targets, tiles of both sizes,
operands in place and laid out."""
import pytest
import torch

import allreduce_reduction_nranks_amd as mrr
from gpu_common import announce
from xent_residue import Targets

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("tokens,rows,cols", [(1, [600, 300], 128), (30, [600, 300], 128), (64, [600, 300], 130),
                                              (65, [600, 300], 128), (200, [600, 300], 130), (700, [40000], 256),
                                              (1500, [900, 3000], 512)])
def test_a_target_s_gradient_has_its_own_rounding_alone(tokens, rows, cols, t):
    announce("xent residue", t, tokens, rows, cols)
    c = Targets(tokens, rows, cols, t, tokens + cols, "cuda")
    dh, dw = torch.empty_like(c.hidden), [torch.empty_like(w) for w in c.weights]
    n = mrr.mrr_linear_xent_workspace_bytes(tokens, cols, rows, len(rows), t, True)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    mrr.check(mrr.mrr_linear_xent_bwd(c.hidden, c.weights, rows, len(rows), c.targets, -100, c.lse, c.dloss, 1, dh, dw, tokens,
                                      cols, cols, cols, t, ws, n))
    torch.cuda.synchronize()
    assert c.share_off(dh, torch.cat(dw)) == [0.0, 0.0]
    for got, (want, tol) in zip((dh, torch.cat(dw)), c.expected()):
        assert bool(((got.double() - want).abs() <= tol).all())
