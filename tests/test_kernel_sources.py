"""Rules that the kernels' sources keep and that no run can show."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_decode_block_gb300", "csrc")


def code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def test_grids_that_start_early_make_no_read_only_loads():
    """A kernel that waits for the grid before it (programmatic dependent launch) lives while that grid still writes:
    a read-only load (ld.global.nc) of what it writes is undefined, and may be moved above the wait.  The append lets
    the next decode start before it has written the rotated queries and the scales."""
    waiting = [f for f in sorted(os.listdir(CSRC)) if f.endswith((".cu", ".cuh")) and "grid_dependency_wait()" in code(f)]
    assert {"pkv_append_tokens.cu", "pkv_attention.cu", "pkv_attention_q8.cu"} <= set(waiting)
    for f in waiting + ["pkv_merge.cuh"]:
        assert not re.search(r"__ldg\b|\.nc\b", code(f)), f
