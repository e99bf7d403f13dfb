"""GPU: bounded-cache calls whose buffers are longer than 32-bit offsets reach
(about 30 GB on the device): records past 4 GB into a cache, query rows past
2^31 elements into a prompt.  Tolerances as in test_gpu_bounded.py."""

import numpy as np
import pytest

import rope_aware_quantized_gb300 as bg
from oracle import bgtq_oracle as O

from tests.test_gpu_bounded import GARBAGE, SCALE, Layer, gather, lens32, zeros_ws
from tests.test_gpu_bounded_many import check_out, check_scores, prompt_plan
from tests.test_gpu_parity import dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [0, 256])
def test_the_last_sequence_of_a_cache_past_4_gb(page):
    B, H, cap, n = 64, 8, 1 << 18, 301
    L = Layer(71, H, 2, 384, 3, [n])
    cache = bg.Cache(L.plan, B, cap, page_tokens=page)
    assert cache.k_codes.numel() > 2 ** 32 + (cap << 9)
    bg.bgtq_quantize_append(L.plan, dev(L.li[0].k[None, :, :n]), dev(L.li[0].v[None, :, :n]),
                            torch.zeros(1, dtype=torch.int32, device="cuda"), cache.sequence_view(B - 1))
    q = torch.zeros((B, 2 * H, 128), dtype=torch.float16, device="cuda")
    q[-1] = dev(L.q[0])
    lens = lens32([0] * (B - 1) + [n])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = [torch.full((B, 2 * H, 128), GARBAGE, device="cuda") for _ in range(2)]
    ws = zeros_ws(bg.bgtq_decode_window_workspace(L.plan, B, n, 4, 100))
    bg.bgtq_decode_window_attn(L.plan, q, cache, lens, n, 4, 100, out[0], ws, status=st)
    scores = torch.full((B, H, cap), GARBAGE, device="cuda")
    scores[-1] = 0
    ws = zeros_ws(bg.bgtq_decode_score_workspace(L.plan, B, n))
    bg.bgtq_decode_score_attn(L.plan, q, cache, lens, n, scores, scores, out[1], ws, status=st)
    dst = bg.Cache(L.plan, B, 64)
    ds, dl = torch.zeros((B, H, 64), device="cuda"), lens32([-7] * B)
    kept = torch.zeros((B, H, 64), dtype=torch.int32, device="cuda")
    bg.bgtq_evict(L.plan, cache, scores, lens, n, 64, 4, 20, dst, ds, dl, kept, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and dl.tolist() == [0] * (B - 1) + [64]
    assert (out[0][:-1] == 0).all() and (out[1][:-1] == 0).all() and (scores[:-1] == GARBAGE).all()
    check_out(L, out[0][-1:].double().cpu().numpy(), lambda m: O.decode_visible(m, 4, 100), False)
    check_out(L, out[1][-1:].double().cpu().numpy(), np.arange, False)
    x = scores[-1:, :, :n + 40].cpu().numpy()
    check_scores(L, x, np.zeros_like(x), np.zeros_like(x), False)
    # the same records as a small cache of this sequence alone, in the order of what stayed
    small = L.cache(n + 1)
    L.fill(small)
    records, after = gather(small, 0, H, n), gather(dst, B - 1, H, 64)
    for h in range(H):
        at = O.evict_positions(x[0, h], n, 64, 4, 20)
        assert np.array_equal(kept[-1, h].cpu().numpy(), at)
        for got, want in zip(after[h], records[h]):
            assert np.array_equal(got, want[at])


def test_a_prompt_past_2_31_elements():
    H, G, T, window = 2, 8, 1050001, 100
    assert H * G * T * 128 > 2 ** 31
    plan = prompt_plan(H, G)
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn((1, H * G, T, 128), device="cuda", dtype=torch.float16, generator=g).mul_(1.5)
    k, v = (torch.randn((1, H, T, 128), device="cuda", dtype=torch.float16, generator=g) for _ in range(2))
    out = torch.full(q.shape, GARBAGE, dtype=torch.float16, device="cuda")
    lse = torch.full(q.shape[:3], GARBAGE, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = bg.Cache(plan, 1, T + 1)
    bg.bgtq_prefill_window_attn(plan, q, k, v, cache, 3, window, out, lse=lse, status=st)
    scores = torch.full((1, H, T), GARBAGE, device="cuda")
    n = bg.bgtq_prefill_score_workspace(plan, 1, T, 0)
    bg.bgtq_prefill_score(plan, q, k, lse, scores, zeros_ws(n), sinks=3, window=window, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for lo in (0, 524288, T - 700):  # rows lo + 400 .. lo + 699 see the sinks and keys of lo + 300 .. lo + 699
        at = torch.cat([torch.arange(3), torch.arange(max(lo, 3), lo + 700)]).cuda()
        i, j = torch.arange(lo, lo + 700, device="cuda")[:, None], at[None, :]
        hidden = ~((j <= i) & ((j < 3) | (j > i - window)))
        for h in range(H):
            rows = slice(h * G, (h + 1) * G)
            qd, kd, vd = q[0, rows, lo:lo + 700].double(), k[0, h, at].double(), v[0, h, at].double()
            s = ((qd @ kd.T) * SCALE).masked_fill(hidden, float("-inf"))
            wlse = torch.logsumexp(s, 2)
            w = torch.exp(s - wlse[..., None])
            d = SCALE * 2.0 ** -17 * (qd.abs() @ kd.abs().T).max().item()
            some = slice(400, 700)
            want = (w @ vd)[:, some]
            tol = (2.0 ** -11 + np.expm1(2 * d) + 2.0 ** -16) * (w @ vd.abs())[:, some] + 128 * 2.0 ** -25 * vd.abs().max()
            tol = tol + 2.0 ** -11 * want.abs() + 2.0 ** -25
            assert ((out[0, rows, lo:lo + 700][:, some].double() - want).abs() <= tol).all(), lo
            assert ((lse[0, rows, lo:lo + 700][:, some].double() - wlse[:, some]).abs()
                    <= d + 2.0 ** -17 + 2.0 ** -21 * wlse[:, some].abs()).all(), lo
            # keys lo + 400 .. lo + 600 (or to the prompt's end) are seen by rows of this block alone
            end = 700 if lo + 700 == T else 601
            cols = (at >= lo + 400) & (at < lo + end)
            ws, wt = w.sum((0, 1))[cols], np.expm1(2 * (2 * d + 2.0 ** -17 + 2.0 ** -20 * wlse.abs().max().item())) + 2.0 ** -17
            assert ((scores[0, h, at[cols]].double() - ws).abs() <= wt * ws + 1e-30).all(), lo
