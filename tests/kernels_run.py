"""Which of the library's kernels a call launches, by torch's profiler: a test that is for one of several kernels that compute
the same says so, and fails where another one runs."""
import re

import torch


def kernels_of(call):
    """The launched kernels' names with their template arguments, such as "qk_walk_k<3, 8, 8, false, true>", in order."""
    from torch.profiler import ProfilerActivity, profile
    torch.cuda.synchronize()
    with profile(activities=[ProfilerActivity.CUDA], acc_events=True) as p:
        call()
        torch.cuda.synchronize()
    names = [re.search(r"mrr::\(anonymous namespace\)::(\w+(?:<[^(]*>)?)", e.name) for e in p.events()]
    return [n.group(1) for n in names if n]


def template_of(name):
    """("qk_walk_k", ["3", "8", "8", "false", "true"]) of such a name."""
    head, _, rest = name.partition("<")
    return head, [a.strip() for a in rest.rstrip(">").split(",")] if rest else []
