"""Kernels that start while the kernel before them still writes (csrc/launch.cuh)
must read their inputs with ordinary loads, behind the wait.

A pointer to const that is also __restrict__ lets the compiler use read-only
loads, which are for memory that nothing writes while the kernel is resident:
such a kernel is resident while its predecessor writes its inputs.  No run
shows it reliably, so the sources are checked.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "context_merge_gb300", "csrc")


def sources():
    """Every file with kernels that launch_early starts, without comments."""
    out = {}
    for name in sorted(os.listdir(CSRC)):
        text = open(os.path.join(CSRC, name)).read()
        if name.endswith(".cu") and '#include "launch.cuh"' in text:
            out[name] = re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)
    return out


def kernels(text):
    """(name, parameters and body) of each __global__ function."""
    parts = re.split(r"__global__", text)[1:]
    for p in parts:
        m = re.search(r"(\w+_kernel)\s*\(", p)
        depth, i = 0, p.index("{", m.end())
        for j in range(i, len(p)):
            depth += (p[j] == "{") - (p[j] == "}")
            if depth == 0:
                yield m.group(1), p[:j]
                break


def test_the_layer_steps_are_covered():
    found = {k for text in sources().values() for k, _ in kernels(text)}
    assert {"glr_fwd_kernel", "glr_bwd_kernel", "glr_step_kernel", "rmsnorm_fwd_kernel", "rmsnorm_bwd_kernel",
            "column_sums_kernel", "wide_kernel", "narrow_kernel", "dz_kernel"} <= found


@pytest.mark.parametrize("name", sorted(sources()))
def test_no_read_only_loads(name):
    text = sources()[name]
    for kernel, body in kernels(text):
        assert "__restrict__" not in body, kernel
        assert "previous_grid_done()" in body, kernel
    for load in ("__ldg", "ld.global.nc", "__ldcv"):
        assert load not in text, load
