"""GPU: bounded-cache calls in combinations: fused steps with a recent-key
buffer, evictions between a paged and a contiguous cache, calls for fewer
sequences than a cache holds.  Tolerances as in test_gpu_bounded.py."""

import numpy as np
import pytest

import rope_aware_quantized_gb300 as bg
from oracle import bgtq_oracle as O

from tests.test_gpu_bounded import (GARBAGE, Layer, bare_layer, check_decode_out, gather, lens32, random_cache, score_call,
                                    score_kinds, window_call, zeros_ws)
from tests.test_gpu_parity import dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("recent,sinks,window", [(20, 4, 40), (64, 8, 40), (300, 30, 50), (2, 0, 1)])
def test_fused_steps_with_a_recent_key_buffer(page, recent, sinks, window):
    L = Layer(81, 2, 3, 384, 3, [300, 41, 1])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ring = []
    for call in ("window", "score"):
        cache = L.cache(304, page, recent)
        L.fill(cache, [n - 1 for n in L.lens])
        if call == "window":
            out = window_call(L, cache, sinks, window, step=True, status=st)
            visible = lambda n: O.decode_visible(n, sinks, window)  # noqa: E731
        else:
            s = torch.zeros((3, 2, 304), device="cuda")
            out = score_call(L, cache, s, s, step=True, status=st)
            visible = np.arange
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        check_decode_out(L, out.double().cpu().numpy(), visible, False, exact_keys=recent)
        ring.append(cache.k_recent)
    for b, n in enumerate(L.lens):
        for h in range(2):
            w = O.attention_weights(L.q[b, 3 * h:3 * h + 3], O.keys_with_recent(L.enc[b][h]["khat"][:n], L.li[b].k[h][:n], recent))
            d = L.logit_error(b, h, np.arange(n))
            tol = (np.expm1(2 * d) + 2.0 ** -16) * w.sum(0) + 2.0 ** -23
            assert (np.abs(s[b, h, :n].double().cpu().numpy() - w.sum(0)) <= tol).all()
    assert torch.equal(*ring)


@pytest.mark.parametrize("src_page,dst_page", [(0, 16), (32, 0), (16, 64)])
def test_evict_between_layouts_and_part_of_a_batch(src_page, dst_page):
    lens, cap, keep, bits, H = [200, 3, 131], 256, 61, (384, 3), 2
    plan = bare_layer(H, *bits).plan
    src, dst = random_cache(plan, H, 5, cap, src_page, bits, 3), random_cache(plan, H, 4, 64, dst_page, bits, 4)
    before = [gather(dst, b, H, 64) for b in range(4)]
    scores = score_kinds("few", (3, H, cap), 5)
    ds, dl = torch.full((3, H, 64), GARBAGE, device="cuda"), lens32([-7] * 3)
    kept = torch.full((3, H, keep), -9, dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    bg.bgtq_evict(plan, src, dev(scores), lens32(lens), 200, keep, 4, 9, dst, ds, dl, kept, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and dl.tolist() == [61, 3, 61]
    for b in range(4):
        after = gather(dst, b, H, 64)
        records = gather(src, b, H, lens[b]) if b < 3 else None
        for h in range(H):
            at = O.evict_positions(scores[b, h], lens[b], keep, 4, 9) if b < 3 else np.zeros(0, int)
            m = len(at)
            if b < 3:
                assert np.array_equal(kept[b, h, :m].cpu().numpy(), at) and (kept[b, h, m:] == -1).all()
                assert np.array_equal(ds[b, h, :m].cpu().numpy(), scores[b, h][at]) and (ds[b, h, m:] == GARBAGE).all()
            for i, (got, old) in enumerate(zip(after[h], before[b][h])):
                assert m == 0 or np.array_equal(got[:m], records[h][i][at])
                assert np.array_equal(got[m:], old[m:])


def test_decode_calls_for_part_of_a_batch():
    L = Layer(82, 2, 2, 256, 2, [90, 33])
    cache = bg.Cache(L.plan, 4, 96)
    L.fill(cache)
    s = torch.full((2, 2, 96), GARBAGE, device="cuda")
    s[0, :, :90] = 0
    s[1, :, :33] = 0
    check_decode_out(L, window_call(L, cache, 4, 20).double().cpu().numpy(), lambda n: O.decode_visible(n, 4, 20), False)
    check_decode_out(L, score_call(L, cache, s, s).double().cpu().numpy(), np.arange, False)
    assert (s[0, :, 90:] == GARBAGE).all() and (s[1, :, 33:] == GARBAGE).all() and (s[1, :, :33] > 0).all()


def test_a_captured_step_replayed_with_growing_lengths_and_no_tokens():
    """One graph of a fused scoring and a windowed step: lengths from an empty sequence on, positions given per replay."""
    n = 40
    L = Layer(83, 1, 4, 384, 3, [n, n])
    cache = L.cache(64)
    kn, vn = (torch.zeros((2, 1, 128), dtype=torch.float16, device="cuda") for _ in range(2))
    pos, lens, q = lens32([0, 0]), lens32([0, 0]), dev(L.q)
    s = torch.full((2, 1, 64), GARBAGE, device="cuda")
    o = [torch.full((2, 4, 128), GARBAGE, device="cuda") for _ in range(2)]
    ws = [zeros_ws(bg.bgtq_decode_score_workspace(L.plan, 2, 64)), zeros_ws(bg.bgtq_decode_window_workspace(L.plan, 2, 64, 2, 9))]

    def step():
        bg.bgtq_decode_score_attn(L.plan, q, cache, lens, 64, s, s, o[0], ws[0], k_new=kn, v_new=vn, pos_new=pos)
        bg.bgtq_decode_window_attn(L.plan, q, cache, lens, 64, 2, 9, o[1], ws[1])

    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        step()
    want = np.zeros((2, 64))
    for i in range(n):
        kn.copy_(dev(np.stack([L.li[b].k[:, i] for b in range(2)])))
        vn.copy_(dev(np.stack([L.li[b].v[:, i] for b in range(2)])))
        pos.fill_(i)
        lens.copy_(lens32([i + 1, 0 if i < 20 else i + 1]))  # (the second one's tokens are appended and not attended at first)
        g.replay()
        torch.cuda.synchronize()
        M = Layer.__new__(Layer)
        M.__dict__.update(L.__dict__, lens=lens.tolist())
        check_decode_out(M, o[0].double().cpu().numpy(), np.arange, False)
        check_decode_out(M, o[1].double().cpu().numpy(), lambda m: O.decode_visible(m, 2, 9), False)
        for b, m in enumerate(M.lens):
            want[b, i] = 0
            if m:
                want[b, :m] += O.attention_weights(L.q[b], L.enc[b][0]["khat"][:m]).sum(0)
            got = s[b, 0].double().cpu().numpy()
            tol = (i + 1) * 4 * (np.expm1(2 * L.logit_error(b, 0, np.arange(n))) + 2.0 ** -16)
            assert (np.abs(got[:i + 1] - want[b, :i + 1]) <= tol).all() and (got[i + 1:] == GARBAGE).all()
            if m == 0:
                assert (got[:i + 1] == 0).all()
