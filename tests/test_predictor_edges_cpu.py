"""The code predictor's operators where calls can go wrong, as far as that shows
without a GPU."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "residual_vector_quantisation_gb300",
                    "csrc")


def kernels(name):
    """(name, parameters, body) of every __global__ function of a source file."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\((?:[^()]|\([^()]*\))*\)\s*)?(\w+)\(([^{]*)\)\s*{", text):
        depth, at = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[at], 0)
            at += 1
        yield m.group(1), m.group(2), text[m.end():at]


@pytest.mark.parametrize("name", ["rvq_norm.cu", "rvq_distill.cu", "rvq_beam.cu"])
def test_overlapping_kernels_take_no_read_only_pointers(name):
    """A kernel that starts while the one before it runs must not promise that what it reads is read-only for its
    whole life: `const ... __restrict__` on a pointer allows loads that are not coherent, and their reordering."""
    found = list(kernels(name))
    assert found
    for kernel, parameters, body in found:
        if "griddep_wait" in body:
            assert "__restrict__" not in parameters and "__ldg(" not in body, kernel
