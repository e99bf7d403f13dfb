"""GPU: the score of a fused scoring step's new position.  It starts from 0
wherever the position lies; the positions next to it stay as they are."""

import numpy as np
import pytest

import rope_aware_quantized_gb300 as bg

from tests.test_gpu_bounded import GARBAGE, Layer, lens32, zeros_ws
from tests.test_gpu_parity import dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

CAP = 64


def call(L, cache, lens, pos, s_in, s_out, max_len, status=None):
    B = len(lens)
    out = torch.zeros((B, L.H * L.G, 128), device="cuda")
    k = dev(np.stack([L.li[b].k[:, 20] for b in range(B)]))
    v = dev(np.stack([L.li[b].v[:, 20] for b in range(B)]))
    bg.bgtq_decode_score_attn(L.plan, dev(L.q), cache, lens32(lens), max_len, s_in, s_out, out,
                              zeros_ws(bg.bgtq_decode_score_workspace(L.plan, B, max_len)), k_new=k, v_new=v,
                              pos_new=lens32(pos), status=status)
    return out


@pytest.mark.parametrize("lens,pos,max_len", [
    ([20, 20, 0], [20, 30, 0], 20),       # at the length, past it, into an empty sequence
    ([20, 20, 0], [63, 19, 5], 64),       # the cache's last position; a position that is attended
    ([0, 0, 0], [0, 1, 2], 0),            # no lengths at all
])
def test_a_new_position_that_is_not_attended_starts_at_zero(lens, pos, max_len):
    L = Layer(61, 2, 3, 384, 3, [24, 24, 24])
    cache = L.cache(CAP)
    L.fill(cache, [20, 20, 20])
    before = np.random.default_rng(1).random((3, 2, CAP)).astype(np.float32) + 1
    for two in (True, False):
        s_in = dev(before)
        s_out = torch.full_like(s_in, GARBAGE) if two else s_in
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        call(L, cache, lens, pos, s_in, s_out, max_len, st)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        got = s_out.cpu().numpy()
        rest = np.full_like(before, GARBAGE) if two else before
        for b, (n, p) in enumerate(zip(lens, pos)):
            for h in range(2):
                x = got[b, h]
                if p >= n:
                    assert x[p] == 0
                else:
                    assert 0 < x[p] <= L.G * (1 + 2.0 ** -20)  # the step's own weights, nothing of what was there
                others = np.array([j for j in range(n, CAP) if j != p])
                assert np.array_equal(x[others], rest[b, h][others])
                mine = np.array([j for j in range(n) if j != p], dtype=int)
                assert (x[mine] >= before[b, h][mine]).all()


def test_a_new_position_outside_the_cache_writes_no_score():
    L = Layer(62, 1, 2, 384, 3, [24, 24])
    cache = L.cache(CAP)
    L.fill(cache, [20, 20])
    s = torch.full((2, 1, CAP), GARBAGE, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    call(L, cache, [0, 0], [-1, CAP], s, s, 20, st)
    torch.cuda.synchronize()
    assert int(st.item()) == bg.STATUS_APPEND_CAPACITY and (s == GARBAGE).all()


def test_a_stale_score_does_not_outlive_a_new_token():
    """A token appended by a step that does not attend it, and attended by the next: its score is its own weights."""
    L = Layer(63, 1, 2, 384, 3, [24])
    cache = L.cache(CAP)
    L.fill(cache, [20])
    s = torch.full((1, 1, CAP), 1000.0, device="cuda")
    s[..., :20] = 0
    call(L, cache, [20], [20], s, s, 20)
    call(L, cache, [21], [21], s, s, 21)
    torch.cuda.synchronize()
    assert s[0, 0, 21].item() == 0 and 0 < s[0, 0, 20].item() <= 2 * (1 + 2.0 ** -20)
    assert (s[0, 0, 22:] == 1000).all()
