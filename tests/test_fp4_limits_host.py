"""Host checks of the 4-bit cache's limits (no GPU: every call below is refused, or its refusal is the next check's)."""

import ctypes as C

import pytest

import rope_aware_quantized_gb300 as bg
from tests.test_rope_fp4_host import call_append, call_attn, fp4, rows


def virtual(capacity, heads):
    """A paged cache with few pages of a large virtual capacity."""
    return fp4(capacity=capacity, heads=heads, page=256, n_pages=8)


@pytest.mark.parametrize("t", [1, 2, 3, 40])
def test_rows_do_not_change_the_limit_on_lengths(t):
    """2048 (sequence, head)s of up to 2^20 positions: as many rows as wanted (past the limits, a workspace too small is what is refused)."""
    c = virtual(1 << 20, 8)
    rc, msg = call_attn(group=8, batch=256, t=t, c=c, max_len=1 << 20, ws_bytes=0)
    assert rc == -4 and "workspace" in msg
    # 2^34 positions in all are one step too many
    rc, msg = call_attn(group=8, batch=256, t=t, c=virtual(1 << 23, 8), max_len=1 << 23, ws_bytes=0)
    assert rc == -2 and "2^34" in msg


def test_an_append_of_more_blocks_than_a_launch_has_is_refused():
    """One row broadcast to 2^30 positions of 4096 heads in a paged cache of as large a virtual capacity."""
    c = virtual(1 << 30, 4096)
    for heads, t, code in ((4096, 1 << 30, -2), (4096, 1 << 25, -2)):
        rc, msg = call_append(c=virtual(1 << 30, heads), t=t, k=rows(sb=0, sh=0, st=0), v=rows(sb=0, sh=0, st=0))
        assert rc == code and "2^31" in msg


def test_sizes_past_64_bits_are_refused_or_right():
    big = (1 << 31) - 1
    for args in ((4096, big, 1 << 30), (4096, 1 << 30, 1 << 30)):  # 2^69 and 2^68 groups
        with pytest.raises(bg.BgtqError, match="64 bits"):
            bg.bgtq_fp4_cache_bytes(*args)
    assert bg.bgtq_fp4_cache_bytes(4096, 1 << 12, 1 << 30) == 2304 << 50  # fits
    # no shape needs more than 304 slots of 256 rows of a workspace: the largest shapes as any large one
    need = bg.bgtq_fp4_attn_workspace(8, 8, 300, 2048, 1 << 20)
    for args in ((4096, 8, big, big, 1 << 30), (4096, 8, 1 << 30, 1 << 30, 1 << 30), (4096, 8, 1 << 29, 1 << 20, 1 << 30), (1, 8, big, big, 1 << 30)):
        assert bg.bgtq_fp4_attn_workspace(*args) == need


def test_a_scale_whose_logits_pass_the_references_range_is_refused():
    """A row's first reference is -1e30: logits below it would get no weight.  |q.k| < 128 * 65504 * 61440 < 2^39, so a scale of 2^40 is safe."""
    for scale in (2.0 ** 40 * (1 + 2.0 ** -23), 1e19, 1e30, 3e38):
        rc, msg = call_attn(scale=scale)
        assert rc == -1 and "softmax_scale" in msg
    rc, msg = call_attn(scale=2.0 ** 40, ws_bytes=0)
    assert rc == -4
