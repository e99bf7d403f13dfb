"""Host check of the eviction's two kernels (no GPU): both start early
(programmatic dependent launch), so what another kernel may still be writing
is read after the wait, and both go by one count of kept positions."""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rope_aware_quantized_gb300", "csrc")


def body(src, kernel):
    """The text of a __global__ function, comments left out."""
    at = src.index("{", src.index(")", src.index("(EvictParams p", src.index(f" {kernel}("))))
    depth = 0
    for i in range(at, len(src)):
        depth += {"{": 1, "}": -1}.get(src[i], 0)
        if depth == 0:
            return re.sub(r"//[^\n]*", "", src[at:i])
    raise AssertionError(kernel)


def test_device_data_is_read_after_the_wait():
    src = open(os.path.join(CSRC, "evict.cu")).read()
    for kernel in ("evict_select_kernel", "evict_move_kernel"):
        before, after = body(src, kernel).split("evict_pdl_wait();")
        # (max_len, keep, cap, H, bk: the launch's own values)
        assert not re.findall(r"evict_len|p\.(?!max_len\b|keep\b|cap\b|H\b|bk\b)\w+", before), kernel
    # one count: the move takes what the selection wrote, not the lengths again
    move = body(src, "evict_move_kernel")
    assert "p.dst_lens[b]" in move and "seq_lens" not in move and "evict_len" not in move
