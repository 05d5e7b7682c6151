"""Tokens to their experts and back, without a GPU."""
import os
import re

from projection_gemm_gb300 import build


def test_rows_written_in_place_are_read_first():
    """Gradients may take y's place, and a store depends on nothing that was read there: what keeps the compiler from
    putting it first is that the loads touch memory."""
    with open(os.path.join(build.CSRC, "skg_experts.cu")) as f:
        loads = re.findall(r'asm volatile\("ld\.global[^;]*;"[^;]*;', f.read())
    assert len(loads) == 4 and all('"memory"' in load for load in loads)
