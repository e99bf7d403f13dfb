"""GPU: an eviction whose lengths come from the kernel right before it, one
that lets its dependents start early: both kernels of the eviction see what
that kernel wrote.  (Records, positions and counts are equal.)"""

import numpy as np
import pytest

import rope_aware_quantized_gb300 as bg
from oracle import bgtq_oracle as O

from tests.test_gpu_bounded import Layer, bare_layer, gather, lens32, random_cache, score_kinds, zeros_ws
from tests.test_gpu_parity import dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

H, CAP, KEEP = 2, 256, 100


def check(src, dst, scores, lens, ds, dl, kept, before):
    """The first len(lens) sequences of dst hold what stays of src."""
    assert dl.tolist() == [min(n, KEEP) for n in lens]
    for b, n in enumerate(lens):
        old, new, records = before[b], gather(dst, b, H, KEEP), gather(src, b, H, n)
        for h in range(H):
            at = O.evict_positions(scores[b, h], n, KEEP, 3, 7)
            m = len(at)
            k = kept[b, h].cpu().numpy()
            assert np.array_equal(k[:m], at) and (k[m:] == -1).all()
            x = ds[b, h].cpu().numpy()
            assert np.array_equal(x[:m], scores[b, h][at]) and (x[m:] == 0).all()
            for got, want, was in zip(new[h], records[h], old[h]):
                assert np.array_equal(got[:m], want[at]) and np.array_equal(got[m:], was[m:])


def buffers(plan, B):
    dst = random_cache(plan, H, B, KEEP, 0, (384, 3), 4)
    return (dst, torch.zeros((B, H, KEEP), device="cuda"), lens32([-7] * B),
            torch.full((B, H, KEEP), -9, dtype=torch.int32, device="cuda"))


def test_lengths_written_by_a_kernel_that_starts_its_dependents_early():
    """A decode writes its outputs over the lengths: as integers a positive float is longer than any sequence (all of
    it), a negative one shorter than none (nothing)."""
    B = 12
    L = Layer(51, 1, 2, 384, 3, [2000])
    cache = L.cache(2000)
    L.fill(cache)
    ws = zeros_ws(bg.bgtq_decode_attn_workspace(L.plan, 1, 2000))
    out = torch.zeros((1, 2, 128), device="cuda")
    lens, now = out.view(torch.int32).view(-1)[:B], lens32([2000])
    P = bare_layer(H, 384, 3).plan
    src = random_cache(P, H, B, CAP, 0, (384, 3), 3)
    scores = score_kinds("spread", (B, H, CAP), 5)
    sd, q = dev(scores), dev(L.q)
    for _ in range(4):
        dst, ds, dl, kept = buffers(P, B)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        before = [gather(dst, b, H, KEEP) for b in range(B)]
        out.zero_()
        torch.cuda.synchronize()
        bg.bgtq_decode_attn(L.plan, q, cache, now, 2000, out, ws)
        bg.bgtq_evict(P, src, sd, lens, CAP, KEEP, 3, 7, dst, ds, dl, kept, status=st)
        torch.cuda.synchronize()
        want = [CAP if x > 0 else 0 for x in out.view(-1)[:B].tolist()]
        assert 0 in want and CAP in want and int(st.item()) == bg.STATUS_SEQLEN_CAPACITY
        check(src, dst, scores, want, ds, dl, kept, before)


def test_lengths_of_an_eviction_feed_the_next():
    B, lens = 3, [256, 40, 170]
    P = bare_layer(H, 384, 3).plan
    src = random_cache(P, H, B, CAP, 0, (384, 3), 6)
    scores = dev(score_kinds("spread", (B, H, CAP), 7))
    mid, two = bg.Cache(P, B, 200), buffers(P, B)
    mid_scores, mid_lens = torch.zeros((B, H, 200), device="cuda"), lens32([0] * B)
    mid_kept = torch.zeros((B, H, 200), dtype=torch.int32, device="cuda")
    dst, ds, dl, kept = two
    before = [gather(dst, b, H, KEEP) for b in range(B)]
    n = lens32(lens)
    torch.cuda.synchronize()
    bg.bgtq_evict(P, src, scores, n, CAP, 200, 3, 7, mid, mid_scores, mid_lens, mid_kept)
    bg.bgtq_evict(P, mid, mid_scores, mid_lens, 200, KEEP, 3, 7, dst, ds, dl, kept)
    torch.cuda.synchronize()
    check(mid, dst, mid_scores.cpu().numpy(), [min(x, 200) for x in lens], ds, dl, kept, before)
