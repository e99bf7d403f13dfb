"""GPU: appends of many groups to the 4-bit cache (the kernel with a warp a group): bytes equal the
oracle's, with and without the rotation, and what is skipped keeps its bytes and sets its status bit."""

import numpy as np
import pytest

import rope_aware_quantized_gb300 as bg
from oracle import rope_fp4_oracle as F
from tests.test_gpu_fp4 import INV, MIXED, check_bytes, group_rows, hard_rows, i32, new_cache, status

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

SECTIONS = [0] * 16 + [1] * 24 + [2] * 24
ROPES = [(0, None), (0, SECTIONS), (1, None), (1, MIXED)]


def many_groups(H, B, T):
    """What chooses the kernel: more than 16 groups a SM."""
    return ((T + 14) // 16 + 1) * H * B > 16 * 152


def put(want, at, p, kc, ks, vc, vs):
    """Position p of the groups `at` (each once) from their rows' codes and scale bytes."""
    for s in (0, 1):
        d = np.arange(s, F.D, 2)
        b = F.KB[p][d]
        want[at[:, None], b] = want[at[:, None], b] & (0xf0 >> 4 * s) | kc[:, d] << 4 * s
    s = p % 2
    want[at[:, None], F.VB[p]] = want[at[:, None], F.VB[p]] & (0xf0 >> 4 * s) | vc << 4 * s
    want[at[:, None], F.KS[p]], want[at[:, None], F.VS[p]] = ks, vs


def expected(before, c, k, v, starts, keep=None):
    """The pool after the append of keys k (rotated) and values v [B][H][T][128] where keep [B][T] says so."""
    want = before.copy().reshape(-1, F.GROUP_BYTES)
    B, H, T, _ = k.shape
    (kc, ks), (vc, vs) = F.fp4_encode(k), F.fp4_encode(v)
    for b in range(B):
        for h in range(H):
            at = group_rows(c, b, h)
            for p in range(16):
                t = np.arange((p - starts[b]) % 16, T, 16)
                t = t if keep is None else t[keep[b][t]]
                if len(t):
                    put(want, at[(starts[b] + t) // 16], p, kc[b, h, t], ks[b, h, t], vc[b, h, t], vs[b, h, t])
    return want


def same(c, want):
    got = c.groups.cpu().numpy().reshape(-1, F.GROUP_BYTES)
    bad = np.argwhere(got != want)
    assert len(bad) == 0, (len(bad), bad[:5], [(got[tuple(i)], want[tuple(i)]) for i in bad[:5]])


def test_the_expected_bytes_are_the_small_appends():
    rng = np.random.default_rng(0)
    k, v = hard_rows(rng, (2, 2, 50, 128)), hard_rows(rng, (2, 2, 50, 128))
    c = new_cache(2, 2, 96, 16, spare=3, seed=1)
    before = c.groups.cpu().numpy()
    bg.bgtq_fp4_append(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), i32([5, 30]), c)
    check_bytes(before, c, k, v, [5, 30])
    same(c, expected(before, c, k, v, [5, 30]))


@pytest.mark.parametrize("B,H,T,cap,page,starts", [
    (2, 8, 2600, 2688, 32, [0, 37]), (1, 2, 19500, 19520, 0, [15]), (40, 3, 321, 352, 16, [(7 * i) % 31 for i in range(40)]),
])
def test_bytes(B, H, T, cap, page, starts):
    assert many_groups(H, B, T)
    rng = np.random.default_rng(T)
    k, v = hard_rows(rng, (B, H, T, 128)), hard_rows(rng, (B, H, T, 128))
    c = new_cache(H, B, cap, page, spare=3, seed=T)
    before = c.groups.cpu().numpy()
    st = status()
    bg.bgtq_fp4_append(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), i32(starts), c, status=st)
    same(c, expected(before, c, k, v, starts))
    assert st.item() == 0


def rotated(k, rope, pos, layout, axis):
    """Keys rotated and rounded to fp16 by the oracle."""
    y = F.rope(k, rope.cos.cpu().numpy(), rope.sin.cpu().numpy(), pos[:, :, None, :], layout, axis)
    return y.astype(np.float16)


@pytest.mark.parametrize("layout,axis", ROPES)
@pytest.mark.parametrize("given", [True, False])
def test_bytes_of_rotated_keys(layout, axis, given):
    B, H, T, starts = 2, 4, 5003, [3, 16]
    assert many_groups(H, B, T)
    rng = np.random.default_rng(layout)
    k, v = hard_rows(rng, (B, H, T, 128)).clip(-40000, 40000), hard_rows(rng, (B, H, T, 128))  # (rotated keys stay finite)
    rope = bg.Rope(*bg.bgtq_rope_table(INV, 6000), layout, axis)
    pos = rng.integers(0, 6000, (rope.axes, B, T)) if given else np.broadcast_to(np.array(starts)[:, None] + np.arange(T), (rope.axes, B, T))
    # rows of a projection: the keys and values of a token side by side
    x = torch.from_numpy(np.concatenate([k, v], 1)).cuda().transpose(1, 2).contiguous()
    c = new_cache(H, B, 5024, 32, spare=3, seed=layout)
    before = c.groups.cpu().numpy()
    st = status()
    bg.bgtq_fp4_append(x[:, :, :H].transpose(1, 2), x[:, :, H:].transpose(1, 2), i32(starts), c, rope=rope,
                       pos=i32(pos) if given else None, status=st)
    same(c, expected(before, c, rotated(k, rope, pos, layout, axis), v, starts))
    assert st.item() == 0


@pytest.mark.parametrize("layout,axis", ROPES)
def test_what_is_skipped_keeps_its_bytes(layout, axis):
    """Of four sequences one past the capacity, one before the start, one onto an unmapped page, and
    positions outside the tables: alone in a group, neighbours that share value bytes, a whole group, the ends."""
    B, H, T, cap = 4, 8, 1301, 1376
    assert many_groups(H, B, T)
    rng = np.random.default_rng(7)
    k, v = (rng.standard_normal((B, H, T, 128)).astype(np.float16) for _ in range(2))
    rope = bg.Rope(*bg.bgtq_rope_table(INV, 2000), layout, axis)
    starts = [11, cap - T + 1, 0, -1]
    pos = rng.integers(0, 2000, (rope.axes, B, T))
    keep = np.ones((B, T), bool)
    keep[[1, 3]] = False
    for b in (0, 2):
        bad = [0, 21, 22, 23, 60, 61, T - 1, *range(5 + 16 * 9, 5 + 16 * 10), *rng.integers(0, T, 40)]
        pos[rng.integers(0, rope.axes, len(bad)), b, bad] = rng.choice([2000, -1, 1 << 30, -(1 << 31)], len(bad))
        keep[b, bad] = False
    c = new_cache(H, B, cap, 32, spare=5, seed=3)
    c.page_table[2, 7] = -1
    c.page_table[2, 30] = c.n_pages
    c.page_table[1] = -1  # (not looked at: nothing of it is appended)
    before = c.groups.cpu().numpy()
    st = status()
    bg.bgtq_fp4_append(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), i32(starts), c, rope=rope, pos=i32(pos), status=st)
    assert st.item() == bg.STATUS_APPEND_CAPACITY | bg.STATUS_ROPE_RANGE | bg.STATUS_PAGE_RANGE
    at = np.arange(T)
    keep[2] &= (at // 32 != 7) & (at // 32 != 30)
    good = np.where((pos >= 0) & (pos < 2000), pos, 0)
    c.page_table[2, 7] = c.page_table[2, 30] = c.page_table[1, 0] = 0  # (no row of theirs is kept)
    c.page_table[1] = 0
    same(c, expected(before, c, rotated(k, rope, good, layout, axis), v, starts, keep))


def test_without_rotation_what_is_skipped_keeps_its_bytes():
    B, H, T, cap = 3, 8, 1800, 1856
    assert many_groups(H, B, T)
    rng = np.random.default_rng(8)
    k, v = (rng.standard_normal((B, H, T, 128)).astype(np.float16) for _ in range(2))
    c = new_cache(H, B, cap, 64, spare=1, seed=4)
    c.page_table[0, 5] = -7
    before = c.groups.cpu().numpy()
    starts, keep, st = [9, 57, 1 << 30], np.ones((B, T), bool), status()
    bg.bgtq_fp4_append(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), i32(starts), c, status=st)
    assert st.item() == bg.STATUS_APPEND_CAPACITY | bg.STATUS_PAGE_RANGE
    keep[0] = (9 + np.arange(T)) // 64 != 5
    keep[1:] = [[False], [False]]  # 57 + 1800 passes the capacity by one
    c.page_table[0, 5] = 0
    same(c, expected(before, c, k, v, starts, keep))
