"""The order of steps at the head of kernels that allocate tensor memory, read from their
sources: what goes wrong otherwise is a grid that waits for good."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fibonacci_spaced_sparse_gb300", "csrc")


def _kernels():
    """(file, text) of every kernel of the library that allocates tensor memory."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        with open(path) as f:
            text = f.read()
        for body in re.split(r"(?=__global__)", text)[1:]:
            if "tc::alloc(" in body:
                yield os.path.basename(path), body


@pytest.mark.parametrize("name,body", list(_kernels()), ids=lambda x: x if x.endswith(".cu") else "")
def test_the_next_launch_starts_behind_the_allocation(name, body):
    """A dependent launch that allocated tensor memory before a CTA of this grid did would
    then wait for this grid, and this CTA for it; so the trigger stands behind the
    allocation and the barrier after it."""
    trigger = body.find("griddepcontrol.launch_dependents")
    if trigger < 0:
        return                             # dependents start when the grid has ended
    alloc = body.index("tc::alloc(")
    barrier = body.index("__syncthreads()", alloc)
    assert alloc < barrier < trigger


def test_there_are_such_kernels():
    assert {name for name, _ in _kernels()} >= {"sfa_fwd_tc.cu", "sfa_qkv.cu", "sfa_qkv_fp8.cu"}
