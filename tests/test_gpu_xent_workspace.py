"""GPU checks that a cross entropy call keeps to the workspace that its size function names, in
place and laid out: what lies behind it is not touched, and both give the same bits."""
import pytest
import torch

import allreduce_reduction_nranks_amd as mrr
from gpu_common import announce

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
GUARD = 1 << 20


@pytest.mark.parametrize("tokens,rows,cols,t", [
    (1, [700, 300], 128, "bf16"), (4, [511], 65, "f16"), (16, [3000, 5], 256, "bf16"), (40, [700, 300], 128, "f16"),
    (64, [4000], 64, "bf16"), (300, [1000, 77], 192, "bf16"), (1000, [513], 1600, "f16"), (130, [1001, 1001, 1001], 520, "f32"),
    (5, [300, 41], 64, "f32"), (700, [2600], 128, "bf16"), (300, [1500], 257, "f16"),
])
def test_nothing_past_the_workspace_is_touched(tokens, rows, cols, t):
    announce("xent workspace", tokens, rows, cols, t)
    g = torch.Generator(device="cuda")
    g.manual_seed(tokens + cols)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    hidden = randn(tokens, cols).to(TYPES[t])
    weights = [(randn(n, cols) / cols ** 0.5).to(TYPES[t]) for n in rows]
    targets = torch.randint(0, sum(rows), (tokens,), generator=g, device="cuda")
    dloss = torch.rand(tokens, generator=g, device="cuda")
    got = []
    for size in (mrr.mrr_linear_xent_workspace_bytes, mrr.mrr_linear_xent_workspace_bytes_in_place):
        loss, lse = torch.empty(tokens, device="cuda"), torch.empty(tokens, device="cuda")
        dh, dw = torch.empty_like(hidden), [torch.empty_like(w) for w in weights]
        for backward in (False, True):
            n = size(tokens, cols, rows, len(rows), t, backward)
            ws = torch.full((n + GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
            if backward:
                mrr.check(mrr.mrr_linear_xent_bwd(hidden, weights, rows, len(rows), targets, -100, lse, dloss, 1, dh, dw, tokens,
                                                  cols, cols, cols, t, ws, n))
            else:
                mrr.check(mrr.mrr_linear_xent_fwd(hidden, weights, rows, len(rows), targets, -100, loss, lse, tokens, cols, cols,
                                                  cols, t, ws, n))
            torch.cuda.synchronize()
            assert bool((ws[n:] == 0xA5).all()), (size.__name__, backward)
        got.append([loss, lse, dh] + dw)
    assert all(torch.equal(a, b) for a, b in zip(*got))
