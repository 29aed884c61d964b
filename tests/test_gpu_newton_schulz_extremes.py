"""GPU checks of mrr_orthogonalize and mrr_muon_step where a call is unusual: norms at the ends of f32, places past 32
bits, the most matrices, the longest, one rank's pointer several times, calls on two streams at once, two graphs with one
workspace."""
import pytest
import torch

import allreduce_reduction_nranks_amd as mrr
from gpu_common import announce
from test_gpu_muon import TYPES, close, exact, gradient, modelled, muon, orth, seeded

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("power", [-149, -140, -120, 100, 120])
@pytest.mark.parametrize("rows,cols", [(20, 30), (90, 140), (140, 90)])
def test_a_power_of_two_does_not_matter(rows, cols, power):
    """Whole numbers of up to 7 bits, times a power of two at which f32 still holds them all: the same bits, as the norm
    divides it out (without eps)."""
    announce("orth power", rows, cols, power)
    g = seeded(rows)
    x = torch.randint(-99, 100, (rows, cols), generator=g, device="cuda").double()
    want, got = torch.empty(rows, cols, device="cuda"), torch.empty(rows, cols, device="cuda")
    mrr.check(orth(x.float(), want, rows, cols, 1, "f32", eps=0.0))
    scaled = (x * 2.0 ** power).float()
    assert torch.equal(scaled.double(), x * 2.0 ** power)
    mrr.check(orth(scaled, got, rows, cols, 1, "f32", eps=0.0))
    assert torch.equal(got, want)
    m, w = torch.empty_like(got), torch.zeros_like(got)
    mrr.check(muon([scaled], 1.0, None, m, 0.0, False, w, [w], -1.0, 0.0, rows, cols, 1, "f32", "f32"))
    assert torch.equal(m, scaled)
    if power > -110:  # (eps, 1e-7, vanishes beside the norm)
        close(w, exact(x), modelled(x, True), 2.0 ** -24, "update")


@pytest.mark.parametrize("way", ["matrices", "rows"])
def test_places_past_32_bits(way):
    announce("orth far", way)
    g = seeded(41)
    batch, rows, cols = 2, 3, 75
    ld, stride = (cols, (1 << 31) + 9) if way == "matrices" else (1 << 31, 100)
    x = gradient(g, batch, rows, cols).bfloat16()
    want, new, m_want = torch.empty_like(x), torch.empty_like(x), torch.empty(batch, rows, cols, device="cuda")
    mrr.check(orth(x, want, rows, cols, batch, "bf16"))
    w0 = torch.randn(batch, rows, cols, generator=g, device="cuda").bfloat16()
    mrr.check(muon([x], 0.5, None, m_want, 0.9, True, w0, [new], 0.02, 0.1, rows, cols, batch, "bf16", "bf16"))

    def far(t):
        return torch.empty((batch - 1) * stride + (rows - 1) * ld + cols, dtype=t, device="cuda").as_strided((batch, rows, cols), (stride, ld, 1))

    src, out, m = far(torch.bfloat16), far(torch.bfloat16), far(torch.float32)
    src.copy_(x)
    mrr.check(orth(src, out, rows, cols, batch, "bf16", ld_in=ld, ld_out=ld, sin=stride, sout=stride))
    assert torch.equal(out, want)
    out.copy_(w0)
    mrr.check(muon([src], 0.5, None, m, 0.9, True, out, [out], 0.02, 0.1, rows, cols, batch, "bf16", "bf16", ld_grad=ld, ld_weight=ld,
                   sg=stride, sw=stride))
    assert torch.equal(out, new) and torch.equal(m, m_want)


@pytest.mark.parametrize("rows,cols", [(1, 1), (2, 3)])
def test_the_most_matrices(rows, cols):
    announce("orth most matrices", rows, cols)
    g = seeded(42)
    batch = 65535
    x = torch.randn(batch, rows, cols, generator=g, device="cuda")
    out, one = torch.empty_like(x), torch.empty(rows, cols, device="cuda")
    mrr.check(orth(x, out, rows, cols, batch, "f32"))
    for k in (0, 1, 255, 32768, 65533, 65534):
        mrr.check(orth(x[k], one, rows, cols, 1, "f32"))
        assert torch.equal(out[k], one)


@pytest.mark.parametrize("rows,cols", [(65536, 3), (65, 65536), (65535, 70)])
@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_the_longest_sides(rows, cols, t):
    announce("orth longest", rows, cols, t)
    g = seeded(43)
    x = gradient(g, rows, cols).to(TYPES[t])
    out = torch.empty_like(x)
    mrr.check(orth(x, out, rows, cols, 1, t))
    close(out, exact(x), modelled(x, t != "bf16" or min(rows, cols) <= 64), torch.finfo(TYPES[t]).eps / 2, "long")


def test_one_rank_several_times_and_a_gradient_for_all_matrices():
    announce("muon one rank several times")
    g = seeded(44)
    rows, cols, batch = 70, 90, 3
    x = gradient(g, rows, cols).bfloat16()
    w = torch.randn(batch, rows, cols, generator=g, device="cuda")
    want, got = ([torch.empty_like(w) for _ in range(3)] for _ in range(2))
    ms = [torch.empty_like(w) for _ in range(2)]
    wide = [x.expand(batch, rows, cols).contiguous() for _ in range(3)]
    mrr.check(muon(wide, 0.25, None, ms[0], 0.9, True, w, want, 0.02, 0.0, rows, cols, batch, "bf16", "f32"))
    mrr.check(muon([x, x, x], 0.25, None, ms[1], 0.9, True, w, got, 0.02, 0.0, rows, cols, batch, "bf16", "f32", sg=0))
    assert torch.equal(ms[0], ms[1]) and all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


def call(seed, rows, cols, t):
    """An update with buffers of its own, and results that do not depend on how often it ran."""
    g = seeded(seed)
    grads = [gradient(g, rows, cols).to(TYPES[t]) for _ in range(2)]
    w = torch.randn(rows, cols, generator=g, device="cuda").to(TYPES[t])
    results = [torch.empty_like(w) for _ in range(2)] + [torch.empty(rows, cols, device="cuda")]
    own = torch.empty(mrr.mrr_muon_workspace_bytes(rows, cols, 1, t), dtype=torch.uint8, device="cuda")

    def run(ws=own):
        mrr.check(muon(grads, 0.5, None, results[2], 0.9, True, w, results[:2], 0.02, 0.0, rows, cols, 1, t, t, ws=ws))
    return run, results


def first_results(calls):
    want = []
    for run, results in calls:
        run()
        torch.cuda.synchronize()
        want.append([r.clone() for r in results])
        for r in results:
            r.zero_()
    torch.cuda.synchronize()
    return want


def test_two_streams_at_once():
    announce("muon two streams")
    calls = [call(45, 300, 700, "bf16"), call(46, 520, 200, "f32")]
    want = first_results(calls)
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(10):
        for s, (run, _) in zip(streams, calls):
            with torch.cuda.stream(s):
                run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for (_, results), w in zip(calls, want) for a, b in zip(results, w))


def test_two_graphs_with_one_workspace():
    announce("muon two graphs")
    calls = [call(47, 300, 700, "bf16"), call(48, 1100, 257, "f16")]
    want = first_results(calls)
    ws = torch.empty(max(mrr.mrr_muon_workspace_bytes(300, 700, 1, "bf16"), mrr.mrr_muon_workspace_bytes(1100, 257, 1, "f16")),
                     dtype=torch.uint8, device="cuda")
    graphs = []
    for run, _ in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run(ws)
        graphs.append(graph)
    for _ in range(3):
        for _, results in calls:
            for r in results:
                r.zero_()
        ws.fill_(255)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for (_, results), w in zip(calls, want) for a, b in zip(results, w))
