"""The ways that the library chooses for the three products of a Newton-Schulz step, read from its planner, and shapes for each way.

A way is (side of a tile, stages in flight, splits of k).  SHAPES: sides of a matrix (either may be its rows), matrices, parts
of an operand, and the ways of A = X X^T, of A^2 and of B X that the planner has for them: every way that any shape of
300000 between 1 and 65536 a side led to, each in one of the smallest that do, with sides that no tile divides.
"""
import ctypes

import allreduce_reduction_nranks_amd as mrr


class _Way(ctypes.Structure):
    _fields_ = [("tile", ctypes.c_uint32), ("stages", ctypes.c_uint32), ("splits", ctypes.c_uint32), ("us", ctypes.c_double)]


class _Plan(ctypes.Structure):
    """mrr::NsPlan of csrc/mrr_ops.hpp."""
    _fields_ = ([(n, _Way) for n in ("gram", "square", "apply")] +
                [(n, ctypes.c_uint32) for n in ("mp", "np", "parts", "m_stages", "n_stages", "counters")] +
                [(n, ctypes.c_uint64) for n in ("x_plane", "o_plane", "x_bytes", "x", "o", "b", "d", "beta", "partial", "part", "counter", "u",
                                                "bytes")])


def plan(rows, cols, batch, parts):
    """The library's plan, mrr::ns_plan(rows, cols, batch, parts, without room for u)."""
    f = mrr.load_library()["_ZN3mrr7ns_planEmmmib"]
    f.restype, f.argtypes = _Plan, [ctypes.c_uint64] * 3 + [ctypes.c_int, ctypes.c_bool]
    return f(rows, cols, batch, parts, False)


def ways(rows, cols, batch, parts):
    p = plan(rows, cols, batch, parts)
    return tuple((w.tile, w.stages, w.splits) for w in (p.gram, p.square, p.apply))


SHAPES = [
    # 11 bits
    ((65, 65), 1, 1, (64, 4, 1), (64, 4, 1), (64, 4, 1)),
    ((129, 2017), 8, 1, (64, 4, 2), (64, 4, 1), (128, 4, 1)),
    ((65, 1944), 1, 1, (64, 4, 4), (64, 4, 1), (64, 4, 1)),
    ((65, 6918), 1, 1, (64, 4, 8), (64, 4, 1), (64, 4, 1)),
    ((193, 202), 64, 1, (128, 4, 1), (128, 4, 1), (128, 4, 1)),
    ((130, 10887), 33, 1, (128, 4, 2), (64, 4, 1), (256, 2, 1)),
    ((129, 29298), 16, 1, (128, 4, 4), (64, 4, 1), (128, 2, 1)),
    ((258, 387), 64, 1, (128, 2, 1), (128, 2, 1), (128, 2, 1)),
    ((130, 7251), 64, 1, (128, 2, 2), (128, 4, 1), (128, 2, 1)),
    ((129, 12161), 33, 1, (128, 2, 4), (64, 4, 1), (128, 2, 1)),
    ((65, 35047), 64, 1, (128, 2, 8), (64, 4, 1), (128, 2, 1)),
    ((2179, 2209), 3, 1, (192, 3, 1), (192, 3, 1), (256, 2, 1)),
    ((387, 389), 64, 1, (256, 2, 1), (256, 2, 1), (256, 2, 1)),
    # two parts
    ((3, 3), 1, 2, (64, 4, 1), (64, 4, 1), (64, 4, 1)),
    ((3, 999), 33, 2, (64, 4, 2), (64, 4, 1), (128, 2, 1)),
    ((3, 962), 1, 2, (64, 4, 4), (64, 4, 1), (64, 4, 1)),
    ((3, 3459), 1, 2, (64, 4, 8), (64, 4, 1), (64, 4, 1)),
    ((193, 202), 64, 2, (128, 4, 1), (128, 4, 1), (128, 4, 1)),
    ((129, 6788), 33, 2, (128, 4, 2), (64, 4, 1), (128, 2, 1)),
    ((129, 24198), 16, 2, (128, 4, 4), (64, 4, 1), (128, 2, 1)),
    ((655, 42768), 1, 2, (128, 4, 8), (64, 4, 1), (128, 2, 1)),
    ((321, 327), 64, 2, (128, 2, 1), (128, 2, 1), (128, 2, 1)),
    ((70, 32433), 128, 2, (128, 2, 4), (64, 4, 1), (128, 2, 1)),
    ((119, 62786), 64, 2, (128, 2, 8), (64, 4, 1), (128, 2, 1)),
    ((2822, 2842), 2, 2, (192, 3, 1), (192, 3, 1), (64, 4, 1)),
]
