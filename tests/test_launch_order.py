"""The order of a kernel's first steps, read from its source: what cannot be provoked
without hanging a GPU."""
import os
import re

import pytest

import sliding_window_learned_b200 as swl

CSRC = os.path.join(os.path.dirname(swl.__file__), "csrc")


def _kernels(path):
    """(name, body) of every __global__ function, comments removed."""
    text = re.sub(r"//[^\n]*", "", open(path).read())
    for m in re.finditer(r"__global__", text):
        head = text.index("{", re.compile(r"\)\s*\{").search(text, m.start()).start())
        depth, i = 1, head + 1
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        name = re.findall(r"(\w+)\s*\(", text[m.start(): head].split("__launch_bounds__")[-1])
        yield [n for n in name if n.endswith("kernel")][0], text[head: i]


def _all():
    return [(f, n, b) for f in sorted(os.listdir(CSRC)) if f.endswith(".cu") for n, b in _kernels(os.path.join(CSRC, f))]


def test_the_kernels_are_found():
    names = {n for _, n, _ in _all()}
    assert {"fwd_tc_kernel", "prior_combine_kernel", "paged_fp8_split_kernel", "cache_append_kernel"} <= names


@pytest.mark.parametrize("name", ["fwd_tc_kernel", "bwd_tc_kernel"])
def test_tensor_memory_is_held_before_a_dependent_may_start(name):
    """A kernel that lets the next one start before it has its tensor memory could wait for
    columns that the next one took, while that one waits for it: the trigger stands
    behind the barrier behind the allocation, inside the branch of the warps that meet there."""
    body = [b for _, n, b in _all() if n == name][0]
    alloc = body.index("tmem_alloc(")
    for m in re.finditer("launch_dependents", body):
        branch = body.index("if (is_tmem_warp", alloc)
        met = body.index("named_barrier_sync(kBarTmem", branch)
        depth = 0
        for ch in body[body.index("{", branch): m.start()]:
            depth += {"{": 1, "}": -1}.get(ch, 0)
        assert alloc < branch < met < m.start() and depth >= 1
