"""GPU checks of every way that the products of a Newton-Schulz step are done: tiles, stages in flight, splits of k, operands in
one part and in two, results as they are and transposed.  Each case is tied to its kernels by name (its splits in
test_product_plans), and held to test_gpu_muon's rounding model."""
import pytest
import torch

import allreduce_reduction_nranks_amd as mrr
from gpu_common import announce
from kernels_run import kernels_of, template_of
from product_plans import SHAPES, ways
from test_gpu_muon import close, exact, gradient, modelled, muon, orth, seeded

pytestmark = pytest.mark.gpu

STEPS = 5


def check_kernels(names, parts, gram, square, apply, turn, short):
    two = str(parts == 2).lower()
    found = {}
    for n in names:
        name, args = template_of(n)
        if name in ("gram_k", "square_k", "apply_k", "short_k"):
            found[(name,) + tuple(args)] = found.get((name,) + tuple(args), 0) + 1
    want = {("apply_k", str(apply[0]), str(apply[1]), two, "false", "false"): STEPS - 1,
            ("apply_k", str(apply[0]), str(apply[1]), two, "true", str(turn).lower()): 1}
    if short:
        want[("short_k", "4", two)] = STEPS
    else:
        want[("gram_k", str(gram[0]), str(gram[1]), two)] = STEPS
        want[("square_k", str(square[0]), str(square[1]), two)] = STEPS
    assert found == want


@pytest.mark.parametrize("tall", [False, True])
@pytest.mark.parametrize("sides,batch,parts,gram,square,apply", SHAPES)
def test_way(sides, batch, parts, gram, square, apply, tall):
    rows, cols = sides[::-1] if tall else sides
    announce("orth way", rows, cols, batch, parts)
    g = seeded(rows + cols)
    x = gradient(g, batch, rows, cols)
    out = torch.full_like(x, float("nan"))
    n = mrr.mrr_orthogonalize_workspace_bytes(rows, cols, batch, "f32", "f16" if parts == 1 else "f32")
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    names = kernels_of(lambda: mrr.check(orth(x, out, rows, cols, batch, "f32", "f16" if parts == 1 else "f32", ws=ws)))
    # (one tile high: A and B in one launch)
    check_kernels(names, parts, gram, square, apply, rows > cols, short=min(sides) <= 64 and apply[0] == 64)
    for k in sorted({0, batch // 2, batch - 1}):
        close(out[k], exact(x[k]), modelled(x[k], parts == 2), 2.0 ** -24, "matrix %d" % k)


@pytest.mark.parametrize("rows,cols,batch,parts", [(4095, 4090, 1, 2), (4090, 4095, 1, 1), (1023, 1021, 4, 2), (1021, 1023, 4, 1),
                                                   (2047, 8190, 1, 1), (8190, 2047, 1, 2), (1600, 1023, 1, 2)])
def test_sides_next_to_those_of_models(rows, cols, batch, parts):
    """As an update, of which all ranks get the result."""
    announce("muon large", rows, cols, batch, parts)
    g = seeded(rows + batch)
    x = gradient(g, batch, rows, cols, noise=0.5).bfloat16()
    w = torch.zeros(batch, rows, cols, device="cuda")
    new, m = [torch.full_like(w, 7.0) for _ in range(2)], torch.empty_like(w)
    products = "f16" if parts == 1 else "auto"
    names = kernels_of(lambda: mrr.check(muon([x, x], 0.5, None, m, 0.0, False, w, new, -1.0, 0.0, rows, cols, batch, "bf16", "f32", products)))
    check_kernels(names, parts, *ways(rows, cols, batch, parts), turn=rows > cols, short=False)
    assert torch.equal(m, x.float()) and torch.equal(new[0], new[1])
    for k in sorted({0, batch - 1}):
        close(new[0][k], exact(x[k]), modelled(x[k], parts == 2), 2.0 ** -24, "matrix %d" % k)
