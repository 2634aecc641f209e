"""When a kernel lets the next one in the stream begin, read from the sources.

A block that has triggered its dependents may find the next kernel's block on
its SM before its own next instruction.  Tensor memory is handed out first
come, first served, and the allocation waits: were the next kernel's block
first, it would hold the columns while it waits for this kernel to end, and
this one would wait for the columns.  So a block's allocation is made, and the
block has met behind it, before any of its threads triggers."""
import glob
import os
import re

import pytest

from transformer_scaled_dot_02_gb300 import build as sd_build

SOURCES = sorted(glob.glob(os.path.join(sd_build.CSRC, "*.cu")))


def _kernels(path):
    """The bodies of a source's kernels, without comments, from each
    __global__ to the next."""
    text = re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path).read(), flags=re.S)
    return text.split("__global__")[1:]


def test_the_kernels_are_found():
    with_tmem = [p for p in SOURCES if any("tmem_alloc(" in k for k in _kernels(p))]
    assert len(with_tmem) >= 6


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_tensor_memory_is_held_before_the_next_kernel_may_begin(path):
    for kernel in _kernels(path):
        alloc, trigger = kernel.find("tmem_alloc("), kernel.find("griddep_launch_dependents()")
        if alloc < 0 or trigger < 0:
            continue
        met = kernel.find("__syncthreads()", alloc)
        assert 0 <= met < trigger
