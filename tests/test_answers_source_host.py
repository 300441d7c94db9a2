"""Order within the tensor-core kernels, read from their sources (no GPU)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(__file__), "..", "autograd_arena_allocated_gb300", "csrc")


@pytest.mark.parametrize("name", ["attn_tc.cu", "gemm_tc_kernel.cuh"])
def test_tensor_memory_is_taken_before_the_next_kernel_may_start(name):
    """A kernel that lets the next one start (pdl_trigger, or pdl_enter, which ends with it) while it has its
    tensor memory still to take may find it taken by a CTA of that next kernel, which waits for this one's end."""
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    found = 0
    for body in text.split("__global__")[1:]:
        alloc = re.search(r"\btmem_alloc\(|tcgen05\.alloc", body)
        if not alloc:
            continue
        found += 1
        starts = [m.start() for m in re.finditer(r"\b(?:pdl_trigger|pdl_enter|enter_after_setup)\b", body)]
        assert starts and min(starts) > alloc.start()
    assert found
