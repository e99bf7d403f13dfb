"""GPU: bounded caches (readings R23-R25) against the oracle: attention with a
sliding window and sinks (one token, a prompt), accumulated attention weights
(one token, a prompt's rows) and eviction, and a run of them together.

Tolerances (derived, not fitted).  A logit is a sum of 128 products: in fp32
its error is at most 128 half-steps, 2^-17 of the sum of the products'
magnitudes; decode also rounds the rotated query to 22 bits.  With d that
bound, a weight exp(s - lse) is off by at most expm1(2 d) of itself plus the
exponential's 2^-21, and an output by that share of sum w |v|.  The prompt's
weights are rounded to fp16 (half a step, 2^-11; below the normal range half
of 2^-24 of the largest) before they meet the values; an fp16 output adds half
a step of itself.  Records, norms, positions and counts are equal.
"""

import numpy as np
import pytest

import rope_aware_quantized_gb300 as bg
from oracle import bgtq_oracle as O
from rope_aware_quantized_gb300 import synth

from tests.test_gpu_parity import dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

SCALE = 1 / np.sqrt(128)
GARBAGE = 7.25  # what untouched floats are filled with


class Layer:
    """A calibrated layer, its sequences' tokens and the oracle's heads."""

    def __init__(self, seed, H, G, bpk, bv, lens):
        self.H, self.G, self.bpk, self.bv, self.lens = H, G, bpk, bv, list(lens)
        n = max(max(lens), 1)
        self.li = [synth.layer_inputs(seed + 31 * b, 0, H, G, n, 1e5, 1.0, n_calib=128) for b in range(len(lens))]
        be = [bg.bgtq_alloc_bits(self.li[0].calib[h], bpk) for h in range(H)]
        self.plan = bg.bgtq_plan_create(np.stack([b for b, _ in be]), np.stack([e for _, e in be]), G, bpk, bv, 77 + seed)
        self.hs = [O.head_state(self.li[0].calib[h], bpk, bv, 77 + seed, h) for h in range(H)]
        self.enc = [[O.encode_head(self.hs[h], l.k[h], l.v[h]) for h in range(H)] for l in self.li]
        # queries of a trained head's spread: logits of a few units
        self.q = np.stack([l.q * np.float16(0.125) for l in self.li])

    def cache(self, cap, page=0, recent=0, seed=5):
        c = bg.Cache(self.plan, len(self.lens), cap, page_tokens=page, recent=recent)
        if page:
            perm = np.random.default_rng(seed).permutation(c.n_pages).astype(np.int32)
            c.page_table.copy_(dev(perm.reshape(c.page_table.shape)))
        return c

    def fill(self, cache, upto=None):
        for b in range(len(self.lens)):
            n = self.lens[b] if upto is None else upto[b]
            if n > 0:
                bg.bgtq_quantize_append(self.plan, dev(self.li[b].k[None, :, :n]), dev(self.li[b].v[None, :, :n]),
                                        torch.zeros(1, dtype=torch.int32, device="cuda"), cache.sequence_view(b))

    def unit(self, b, h, g):
        return self.q[b, h * self.G + g]

    def logit_error(self, b, h, keys):
        """Bound of a logit's error, from the sum of the products' magnitudes (by norms in the codec's own domain)."""
        q = self.q[b, h * self.G:(h + 1) * self.G].astype(np.float64)
        e, kc = self.enc[b][h], self.hs[h].kc
        y = O.dequant(e["kcodes"], e["krho"], kc, codec_domain=True).astype(np.float64)
        qc = q[:, kc.perm] * kc.sig.astype(np.float64)  # an orthogonal rotation of it meets y
        mag = np.linalg.norm(qc, axis=1).max() * np.linalg.norm(y[keys], axis=1).max() if len(keys) else 0.0
        # (the recent-key buffer's logits: the products of the keys as given)
        mag = max(mag, (np.abs(q) @ np.abs(self.li[b].k[h].astype(np.float64)).T).max())
        return SCALE * mag * (2.0 ** -17 + 2.0 ** -22)


def lens32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def zeros_ws(n):
    return torch.zeros(max(n, 16), dtype=torch.uint8, device="cuda")


def check_decode_out(L, got, visible, half, exact_keys=None):
    """out [B][H*G][128] against the oracle's attention over each sequence's visible positions."""
    for b, n in enumerate(L.lens):
        at = visible(n)
        for h in range(L.H):
            e = L.enc[b][h]
            k = e["khat"][:n].astype(np.float64)
            if exact_keys:
                k = O.keys_with_recent(e["khat"][:n], L.li[b].k[h][:n], exact_keys)
            rows = slice(h * L.G, (h + 1) * L.G)
            if n == 0:
                assert (got[b, rows] == 0).all()
                continue
            w = O.attention_weights(L.q[b, rows], k[at])
            v = e["vhat"][at].astype(np.float64)
            want, d = w @ v, L.logit_error(b, h, at)
            # weights off by expm1(2 d) + 2^-21; P' = p rho_V as hi + lo keeps 22 bits, sums 2^-17.
            # The sum runs over the value codec's coordinates o_j, each rounded relative to
            # itself (2^-22 by P', 2^-23 a sum); the inverse rotation then adds 128 of them
            # with weights +-1/sqrt(128) in 7 rounded stages, so a dim that cancels keeps an
            # error of up to 2^-20 sum |o_j| / sqrt(128) <= 2^-20 |o| <= 2^-20 max |v_t|.
            tol = (np.expm1(2 * d) + 2.0 ** -16) * (w @ np.abs(v)) + 2.0 ** -20 * np.linalg.norm(v, axis=1).max()
            if half:
                tol = tol + 2.0 ** -11 * np.abs(want) + 2.0 ** -25
            assert (np.abs(got[b, rows] - want) <= tol).all(), (b, h, np.abs(got[b, rows] - want).max(), tol.min())


def window_call(L, cache, sinks, window, half=False, step=False, max_len=None, status=None, stream=None, ws=None):
    B = len(L.lens)
    out = torch.full((B, L.H * L.G, 128), GARBAGE, dtype=torch.float16 if half else torch.float32, device="cuda")
    max_len = max(L.lens) if max_len is None else max_len
    ws = zeros_ws(bg.bgtq_decode_window_workspace(L.plan, B, max_len, sinks, window)) if ws is None else ws
    new = {}
    if step:
        at = [max(n - 1, 0) for n in L.lens]
        new = dict(k_new=dev(np.stack([L.li[b].k[:, at[b]] for b in range(B)])),
                   v_new=dev(np.stack([L.li[b].v[:, at[b]] for b in range(B)])), pos_new=lens32(at))
    bg.bgtq_decode_window_attn(L.plan, dev(L.q), cache, lens32(L.lens), max_len, sinks, window, out, ws, status=status,
                               stream=stream, **new)
    return out


WINDOW_CASES = [
    # lens, sinks, window, page, half, step, (bpk, bv), (H, G)
    ([200], 4, 33, 0, False, False, (384, 3), (1, 4)),
    ([1], 4, 33, 0, False, False, (384, 3), (1, 4)),
    ([1, 0, 17, 300], 0, 1, 0, False, False, (256, 2), (2, 3)),
    ([1, 0, 17, 300], 1, 16, 16, True, False, (256, 2), (2, 8)),
    ([129, 128, 127], 16, 112, 16, False, True, (384, 2), (2, 1)),
    ([300, 299, 64, 65], 17, 47, 32, True, True, (128, 3), (2, 7)),
    ([500], 40, 500, 0, False, True, (384, 4), (1, 8)),     # the window covers everything
    ([500], 1000, 3, 64, False, False, (384, 1), (1, 2)),   # the sinks cover everything
    ([1700, 33], 5, 1029, 0, False, True, (384, 3), (2, 8)),
    ([2500], 100, 1200, 256, False, True, (128, 1), (1, 4)),
]


@pytest.mark.parametrize("lens,sinks,window,page,half,step,bits,hg", WINDOW_CASES)
def test_decode_window(lens, sinks, window, page, half, step, bits, hg):
    L = Layer(3, hg[0], hg[1], bits[0], bits[1], lens)
    cap = -(-max(lens) // max(page, 2)) * max(page, 2) + max(page, 2)
    cache = L.cache(cap, page)
    L.fill(cache, [max(n - 1, 0) for n in lens] if step else None)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    if page:  # pages without a visible position are unmapped
        pt = cache.page_table.cpu().numpy().copy()
        for b, n in enumerate(lens):
            used = {j // page for j in O.decode_visible(n, sinks, window)} | ({max(n - 1, 0) // page} if step else set())
            for i in range(pt.shape[1]):
                if i not in used:
                    pt[b, i] = -1
        cache.page_table.copy_(dev(pt))
    out = window_call(L, cache, sinks, window, half, step, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    check_decode_out(L, out.double().cpu().numpy(), lambda n: O.decode_visible(n, sinks, window), half)


def test_decode_window_as_long_as_the_sequence_is_plain_decode_bit_for_bit():
    L = Layer(4, 2, 8, 384, 3, [700, 1300, 5])
    cache = L.cache(1400)
    L.fill(cache)
    ws = zeros_ws(bg.bgtq_decode_attn_workspace(L.plan, 3, 1300))
    want = torch.empty((3, 16, 128), dtype=torch.float32, device="cuda")
    bg.bgtq_decode_attn(L.plan, dev(L.q), cache, lens32(L.lens), 1300, want, ws)
    assert torch.equal(window_call(L, cache, 0, 1300), want)
    assert torch.equal(window_call(L, cache, 3, 5000), want)


def test_decode_window_with_a_recent_key_buffer():
    for recent, sinks, window in ((20, 4, 40), (64, 8, 40), (300, 30, 50), (500, 600, 1)):
        L = Layer(5, 1, 4, 384, 3, [500])
        cache = L.cache(600, recent=recent)
        L.fill(cache)
        out = window_call(L, cache, sinks, window, step=False)
        torch.cuda.synchronize()
        # the exact keys' logits are fp16 products: at most the packed ones' bound with the norms of the keys as given
        check_decode_out(L, out.double().cpu().numpy(), lambda n: O.decode_visible(n, sinks, window), False, exact_keys=recent)


def test_decode_window_reports_lengths_and_pages():
    L = Layer(6, 1, 2, 384, 3, [100])
    cache = L.cache(128, page=16)
    L.fill(cache)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    long = Layer.__new__(Layer)
    long.__dict__.update(L.__dict__, lens=[1000])
    out = window_call(long, cache, 4, 8, max_len=100, status=st)  # cut to max_len
    torch.cuda.synchronize()
    assert int(st.item()) == bg.STATUS_SEQLEN_CAPACITY
    check_decode_out(L, out.double().cpu().numpy(), lambda n: O.decode_visible(n, 4, 8), False)
    st.zero_()
    cache.page_table[0, 0] = -1  # the sinks' page
    window_call(L, cache, 4, 8, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == bg.STATUS_PAGE_RANGE
    st.zero_()
    window_call(L, cache, 0, 8, status=st)  # no sinks: that page is not read
    torch.cuda.synchronize()
    assert int(st.item()) == 0


def score_call(L, cache, s_in, s_out, half=False, step=False, status=None, max_len=None, ws=None, stream=None):
    B = len(L.lens)
    out = torch.full((B, L.H * L.G, 128), GARBAGE, dtype=torch.float16 if half else torch.float32, device="cuda")
    max_len = max(L.lens) if max_len is None else max_len
    ws = zeros_ws(bg.bgtq_decode_score_workspace(L.plan, B, max_len)) if ws is None else ws
    new = {}
    if step:
        at = [max(n - 1, 0) for n in L.lens]
        new = dict(k_new=dev(np.stack([L.li[b].k[:, at[b]] for b in range(B)])),
                   v_new=dev(np.stack([L.li[b].v[:, at[b]] for b in range(B)])), pos_new=lens32(at))
    bg.bgtq_decode_score_attn(L.plan, dev(L.q), cache, lens32(L.lens), max_len, s_in, s_out, out, ws, status=status,
                              stream=stream, **new)
    return out


def want_scores(L, before, after, step):
    """Expected scores and their tolerance."""
    want, tol = after.copy(), np.zeros_like(after)
    for b, n in enumerate(L.lens):
        for h in range(L.H):
            if n == 0:
                continue
            w = O.attention_weights(L.q[b, h * L.G:(h + 1) * L.G], L.enc[b][h]["khat"][:n]).sum(0)
            was = before[b, h, :n].copy()
            if step:
                was[n - 1] = 0
            want[b, h, :n] = was + w
            tol[b, h, :n] = (np.expm1(2 * L.logit_error(b, h, np.arange(n))) + 2.0 ** -17) * w + 2.0 ** -23 * np.abs(was + w)
    return want, tol


@pytest.mark.parametrize("lens,page,half,step,bits,hg", [
    ([200], 0, False, False, (384, 3), (1, 4)),
    ([1], 0, False, True, (384, 3), (1, 4)),
    ([1, 0, 17, 300], 0, False, False, (256, 2), (2, 3)),
    ([1, 0, 17, 300], 16, True, False, (256, 2), (2, 8)),
    ([129, 128, 127], 16, False, True, (384, 2), (2, 1)),
    ([1700, 33], 0, False, True, (384, 3), (2, 7)),
    ([2501], 64, True, True, (128, 4), (1, 8)),
])
def test_decode_score(lens, page, half, step, bits, hg):
    L = Layer(8, hg[0], hg[1], bits[0], bits[1], lens)
    cap = -(-max(lens) // max(page, 2)) * max(page, 2) + max(page, 2)
    cache = L.cache(cap, page)
    L.fill(cache, [max(n - 1, 0) for n in lens] if step else None)
    before = np.random.default_rng(1).random((len(lens), L.H, cap)).astype(np.float32)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    two = torch.full(before.shape, GARBAGE, device="cuda")
    out = score_call(L, cache, dev(before), two, half, step, st)
    one = dev(before)
    out1 = score_call(L, cache, one, one, half, step, st)  # in place
    plain = torch.empty_like(out)
    bg.bgtq_decode_attn(L.plan, dev(L.q), cache, lens32(lens), max(lens), plain,
                        zeros_ws(bg.bgtq_decode_attn_workspace(L.plan, len(lens), max(lens))))
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert torch.equal(out, plain) and torch.equal(out1, plain)
    check_decode_out(L, out.double().cpu().numpy(), np.arange, half)
    for got, rest in ((two, np.full_like(before, GARBAGE)), (one, before)):
        want, tol = want_scores(L, before.astype(np.float64), rest.astype(np.float64), step)
        x = got.double().cpu().numpy()
        assert (np.abs(x - want) <= tol).all(), np.abs(x - want).max()
        for b, n in enumerate(lens):
            assert np.array_equal(x[b, :, n:], rest[b, :, n:])  # behind the sequence: as they were
    # the same bits on every run
    again = dev(before)
    score_call(L, cache, again, again, half, step, st)
    assert torch.equal(again, one)


def test_decode_score_with_a_recent_key_buffer_and_long_lengths():
    L = Layer(9, 1, 4, 384, 3, [300])
    cache = L.cache(320, recent=32)
    L.fill(cache)
    s = torch.zeros((1, 1, 320), device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    long = Layer.__new__(Layer)
    long.__dict__.update(L.__dict__, lens=[100000])
    out = score_call(long, cache, s, s, status=st, max_len=300)
    torch.cuda.synchronize()
    assert int(st.item()) == bg.STATUS_SEQLEN_CAPACITY
    check_decode_out(L, out.double().cpu().numpy(), np.arange, False, exact_keys=32)
    k = O.keys_with_recent(L.enc[0][0]["khat"], L.li[0].k[0], 32)
    w = O.attention_weights(L.q[0], k).sum(0)
    tol = (np.expm1(2 * L.logit_error(0, 0, np.arange(300))) + 2.0 ** -16) * w + 2.0 ** -23
    assert (np.abs(s[0, 0, :300].double().cpu().numpy() - w) <= tol).all()
    assert (s[0, 0, 300:] == 0).all()


def prompt(L, seed=2):
    """Queries [B][H*G][T][128] of a few units' logits, K and V of each sequence (all of one length)."""
    T = max(L.lens)
    r = np.random.default_rng(seed)
    q = np.stack([np.concatenate([l.k[h][r.permutation(T)][None] * np.float16(0.125) for h in range(L.H) for _ in range(L.G)])
                  for l in L.li]).astype(np.float16)
    return q, np.stack([l.k[:, :T] for l in L.li]), np.stack([l.v[:, :T] for l in L.li])


def prompt_logit_error(q, k):
    return SCALE * 2.0 ** -17 * (np.abs(q.astype(np.float64)) @ np.abs(k.astype(np.float64)).T).max()


@pytest.mark.parametrize("T,B,sinks,window,half,bits,hg", [
    (1, 1, 4, 8, False, (384, 3), (1, 4)),
    (77, 2, 0, 1, True, (384, 3), (2, 3)),
    (128, 1, 5, 64, False, (256, 2), (1, 8)),
    (129, 1, 0, 128, True, (256, 2), (2, 1)),
    (300, 2, 17, 25, False, (384, 2), (1, 4)),
    (513, 1, 130, 127, True, (128, 4), (2, 7)),
    (700, 1, 4, 129, False, (384, 3), (1, 2)),
    (640, 1, 200, 300, True, (384, 3), (1, 5)),
    (385, 1, 400, 1, False, (384, 3), (1, 4)),      # the sinks cover the prompt
    (600, 1, 0, 10000, True, (384, 3), (2, 8)),     # no window
])
def test_prefill_window(T, B, sinks, window, half, bits, hg):
    L = Layer(11, hg[0], hg[1], bits[0], bits[1], [T] * B)
    q, k, v = prompt(L)
    cap = T + T % 2 + 2
    cache, plain = L.cache(cap), L.cache(cap)
    for c in (cache, plain):
        for x in (c.k_codes, c.v_codes):
            x.fill_(0xA5)
    out = torch.full(q.shape, GARBAGE, dtype=torch.float16 if half else torch.float32, device="cuda")
    lse = torch.full(q.shape[:3], GARBAGE, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    bg.bgtq_prefill_window_attn(L.plan, dev(q), dev(k), dev(v), cache, sinks, window, out, lse=lse, status=st)
    ref = torch.empty_like(out)
    bg.bgtq_prefill_attn(L.plan, dev(q), dev(k), dev(v), plain, ref)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for n in ("k_codes", "v_codes", "k_norm", "v_norm"):
        assert torch.equal(getattr(cache, n), getattr(plain, n)), n
    out2 = torch.empty_like(out)
    bg.bgtq_prefill_window_attn(L.plan, dev(q), dev(k), dev(v), cache, sinks, window, out2)  # without lse
    assert torch.equal(out, out2)
    for b in range(B):
        for h in range(L.H):
            rows = slice(h * L.G, (h + 1) * L.G)
            want, wlse, w = O.prefill_window(q[b, rows], k[b, h], v[b, h], sinks, window)
            d = max(prompt_logit_error(q[b, i], k[b, h]) for i in range(rows.start, rows.stop))
            va = np.abs(v[b, h].astype(np.float64))
            tol = (2.0 ** -11 + np.expm1(2 * d) + 2.0 ** -16) * np.einsum("gij,jd->gid", w, va) + T * 2.0 ** -25 * va.max()
            if half:
                tol = tol + 2.0 ** -11 * np.abs(want) + 2.0 ** -25
            got = out[b, rows].double().cpu().numpy()
            assert (np.abs(got - want) <= tol).all(), (b, h, np.abs(got - want).max())
            dl = np.abs(lse[b, rows].double().cpu().numpy() - wlse)
            assert (dl <= d + 2.0 ** -17 + 2.0 ** -21 * np.abs(wlse)).all(), dl.max()


@pytest.mark.parametrize("T,B,row0,sinks,window,hg", [
    (1, 1, 0, 0, 1, (1, 4)),
    (77, 2, 0, 0, 77, (2, 3)),
    (300, 1, 0, 0, 300, (1, 8)),
    (300, 2, 290, 0, 300, (2, 7)),       # ten rows: eight heads' rows in a tile
    (300, 1, 299, 4, 20, (1, 5)),        # one row
    (385, 1, 321, 0, 385, (2, 4)),       # 64 rows: two heads' rows in a tile
    (385, 1, 300, 0, 385, (1, 2)),       # 85 rows
    (385, 1, 385, 0, 385, (1, 2)),       # none
    (640, 1, 100, 17, 129, (1, 4)),
    (515, 1, 0, 130, 64, (1, 3)),
    (1300, 1, 0, 4, 1300, (1, 8)),       # query heads shared out over CTAs
    (1300, 2, 37, 0, 200, (2, 3)),       # and row tiles, under a window
    (2100, 1, 0, 0, 2100, (1, 1)),       # row tiles alone
])
def test_prefill_score(T, B, row0, sinks, window, hg):
    L = Layer(12, hg[0], hg[1], 384, 3, [T] * B)
    q, k, _ = prompt(L)
    lse = np.full(q.shape[:3], np.nan, np.float32)  # rows before row0 are not read
    want = np.zeros((B, L.H, T))
    tol = np.zeros_like(want)
    for b in range(B):
        for h in range(L.H):
            rows = slice(h * L.G, (h + 1) * L.G)
            _, wlse, w = O.prefill_window(q[b, rows], k[b, h], k[b, h], sinks, window)
            lse[b, rows, row0:] = wlse[:, row0:]
            want[b, h] = w[:, row0:].sum((0, 1))
            d = max(prompt_logit_error(q[b, i], k[b, h]) for i in range(rows.start, rows.stop))
            d += 2.0 ** -22 * np.abs(wlse).max()  # lse and its product with log2 e in fp32
            tol[b, h] = (np.expm1(2 * d) + 2.0 ** -17) * want[b, h] + 1e-30
    stride = T + 3
    scores = torch.full((B, L.H, stride), GARBAGE, device="cuda")
    n = bg.bgtq_prefill_score_workspace(L.plan, B, T, row0)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(row0=row0, sinks=sinks, window=window, status=st)
    bg.bgtq_prefill_score(L.plan, dev(q), dev(k), dev(lse), scores, ws, **kw)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    got = scores.double().cpu().numpy()
    assert (got[:, :, T:] == GARBAGE).all()
    assert (np.abs(got[:, :, :T] - want) <= tol).all(), (np.abs(got[:, :, :T] - want).max(), tol.max())
    if T == 300 and row0 == 0:  # a row that saw nothing gives nothing
        lse[:, :, 5] = -np.inf
        other = torch.empty_like(scores)
        bg.bgtq_prefill_score(L.plan, dev(q), dev(k), dev(lse), other, ws, **kw)
        for b in range(B):
            for h in range(L.H):
                _, _, w = O.prefill_window(q[b, h * L.G:(h + 1) * L.G], k[b, h], k[b, h], sinks, window)
                x = other[b, h, :T].double().cpu().numpy()
                assert (np.abs(x - (want[b, h] - w[:, 5].sum(0))) <= tol[b, h] + 1e-6).all()


def evict_reference(L, cap, lens, scores, keep, sinks, recent, records):
    """Expected kept positions, scores and records [B][H] of a cache holding `records`."""
    out = {}
    for b, n in enumerate(lens):
        for h in range(L.H):
            at = O.evict_positions(scores[b, h], n, keep, sinks, recent)
            kc, kn, vc, vn = records[b][h]
            out[b, h] = (at, scores[b, h][at], kc[at], kn[at], vc[at], vn[at])
    return out


def gather(cache, b, H, n):
    """Per head (K records, key norms, V codes, value norms) of positions 0 .. n-1 of sequence b."""
    pt = cache.page_table.cpu().numpy() if cache.page_table is not None else None
    P = cache.page_tokens
    rec = []
    kr = cache.k_codes.cpu().numpy()
    vr = cache.v_codes.cpu().numpy()
    kn, vn = cache.k_norm.cpu().numpy(), cache.v_norm.cpu().numpy()
    pos = np.arange(n + n % 2)
    for h in range(H):
        slot = (b * H + h) * cache.capacity + pos if pt is None else (pt[b, pos // P].astype(np.int64) * H + h) * P + pos % P
        slots = len(kn)
        k = kr.reshape(slots, -1)[slot[:n]]
        vrec = vr.reshape(slots // 2, -1)[slot[::2] // 2]
        bv = vrec.shape[1] // 32
        rec.append((k, kn[slot[:n]], O.unpack_v(vrec, bv, len(pos))[:n] if n else np.zeros((0, 128), np.int64), vn[slot[:n]]))
    return rec


def random_cache(plan, H, B, cap, page, bits, seed):
    """A cache of random records (eviction does not look into them)."""
    c = bg.Cache(plan, B, cap, page_tokens=page)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    for x in (c.k_codes, c.v_codes):
        x.copy_(torch.randint(0, 256, x.shape, device="cuda", generator=g, dtype=torch.int32).to(torch.uint8))
    for x in (c.k_norm, c.v_norm):
        x.copy_(torch.rand(x.shape, device="cuda", generator=g))
    if page:
        perm = np.random.default_rng(seed).permutation(c.n_pages).astype(np.int32)
        c.page_table.copy_(dev(perm.reshape(c.page_table.shape)))
    return c


def bare_layer(H, bpk, bv):
    L = Layer.__new__(Layer)
    L.H, L.G, L.bpk, L.bv = H, 2, bpk, bv
    L.plan = bg.bgtq_plan_create(np.full((H, 64), bpk // 128, np.uint8), np.ones((H, 64)), 2, bpk, bv, 1)
    return L


def score_kinds(kind, shape, seed):
    r = np.random.default_rng(seed)
    if kind == "spread":
        return np.exp(2 * r.standard_normal(shape)).astype(np.float32)
    if kind == "equal":
        return np.full(shape, 0.5, np.float32)
    if kind == "few":  # many ties
        return r.integers(0, 4, shape).astype(np.float32)
    x = r.standard_normal(shape).astype(np.float32)  # signs, zeros of both signs, infinities, NaN
    for i, v in enumerate((0.0, -0.0, np.inf, -np.inf, np.nan)):
        x[r.random(shape) < 0.06 * (i + 1) / 3] = v
    return x


@pytest.mark.parametrize("lens,cap,page,keep,sinks,recent,bits,kind", [
    ([100], 128, 0, 10, 2, 3, (384, 3), "spread"),
    ([100], 128, 0, 11, 0, 0, (384, 3), "equal"),
    ([100], 128, 0, 1, 0, 0, (128, 1), "odd"),
    ([100, 0, 1, 37, 36], 128, 0, 37, 4, 8, (256, 2), "odd"),
    ([100, 0, 1, 37, 36], 128, 16, 37, 4, 8, (256, 2), "few"),
    ([200, 131], 256, 32, 50, 20, 30, (384, 5), "spread"),   # the always-kept fill the budget
    ([200, 131], 256, 0, 129, 0, 129, (512, 4), "few"),
    ([4095, 4097, 3000], 4100, 0, 1025, 4, 64, (384, 3), "odd"),
    ([9001, 5000], 9216, 64, 4000, 16, 100, (384, 2), "few"),
    ([40001], 40002, 0, 20001, 0, 1, (128, 3), "spread"),
    ([40001], 40002, 0, 200, 7, 0, (128, 1), "equal"),
    ([300001], 300002, 0, 1001, 4, 10, (128, 1), "few"),     # segments longer than their shared memory
])
def test_evict(lens, cap, page, keep, sinks, recent, bits, kind):
    H, B = (1 if cap > 50000 else 2), len(lens)
    L = bare_layer(H, *bits)
    src = random_cache(L.plan, H, B, cap, page, bits, 3)
    dcap = -(-min(keep, max(lens)) // max(page, 2)) * max(page, 2)
    dst = random_cache(L.plan, H, B, dcap, page, bits, 4)
    before = [gather(dst, b, H, dcap) for b in range(B)]
    scores = score_kinds(kind, (B, H, cap), 5)
    ds = torch.full((B, H, dcap), GARBAGE, device="cuda")
    dl = lens32([-7] * B)
    kept = torch.full((B, H, keep), -9, dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    bg.bgtq_evict(L.plan, src, dev(scores), lens32(lens), max(lens), keep, sinks, recent, dst, ds, dl, kept, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    records = [gather(src, b, H, lens[b]) for b in range(B)]
    want = evict_reference(L, cap, lens, scores, keep, sinks, recent, records)
    assert dl.tolist() == [min(n, keep) for n in lens]
    for b in range(B):
        after = gather(dst, b, H, dcap)
        for h in range(H):
            at, sc, kc, kn, vc, vn = want[b, h]
            m = len(at)
            k = kept[b, h].cpu().numpy()
            assert np.array_equal(k[:m], at) and (k[m:] == -1).all()
            x = ds[b, h].cpu().numpy()
            assert np.array_equal(x[:m], sc, equal_nan=True) and (x[m:] == GARBAGE).all()
            for got, w, old in zip(after[h], (kc, kn, vc, vn), before[b][h]):
                assert np.array_equal(got[:m], w) and np.array_equal(got[m:], old[m:])


def test_evict_within_one_pool():
    """Source and destination share the pools of pages; their page tables share no page."""
    L = bare_layer(2, 384, 3)
    src = random_cache(L.plan, 2, 1, 256, 16, (384, 3), 6)
    dst = bg.Cache(L.plan, 1, 64, page_tokens=16)
    src.page_table.copy_(dev(np.arange(16, dtype=np.int32)[None, ::-1].copy()))
    # positions 160 .. 255 are not in use: their pages (5 .. 0) hold the destination
    dst.page_table.copy_(lens32([[5, 2, 0, 3]]))
    for n in ("k_codes", "v_codes", "k_norm", "v_norm"):
        setattr(dst, n, getattr(src, n))
    dst.n_pages = src.n_pages
    dst.desc = dst._desc(0, 0, 0, 0, 0)
    records = [gather(src, 0, 2, 160)]
    scores = score_kinds("spread", (1, 2, 256), 7)
    ds, dl = torch.zeros((1, 2, 64), device="cuda"), lens32([0])
    kept = torch.zeros((1, 2, 63), dtype=torch.int32, device="cuda")
    bg.bgtq_evict(L.plan, src, dev(scores), lens32([160]), 160, 63, 4, 9, dst, ds, dl, kept)
    torch.cuda.synchronize()
    want = evict_reference(L, 256, [160], scores, 63, 4, 9, records)
    after = gather(dst, 0, 2, 63)
    for h in range(2):
        assert np.array_equal(kept[0, h].cpu().numpy(), want[0, h][0])
        for got, w in zip(after[h], want[0, h][2:]):
            assert np.array_equal(got, w)


def test_evict_reports_lengths_and_pages():
    L = bare_layer(1, 384, 3)
    src = random_cache(L.plan, 1, 2, 64, 16, (384, 3), 8)
    dst = bg.Cache(L.plan, 2, 16)
    scores = score_kinds("spread", (2, 1, 64), 9)
    ds, dl = torch.zeros((2, 1, 16), device="cuda"), lens32([0, 0])
    kept = torch.zeros((2, 1, 16), dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    bg.bgtq_evict(L.plan, src, dev(scores), lens32([-3, 99]), 50, 16, 0, 4, dst, ds, dl, kept, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == bg.STATUS_SEQLEN_CAPACITY and dl.tolist() == [0, 16]
    assert np.array_equal(kept[1, 0].cpu().numpy(), O.evict_positions(scores[1, 0], 50, 16, 0, 4))
    st.zero_()
    src.page_table[1, 2] = 1000  # positions 32 .. 47; the last four kept positions are 46 .. 49
    bg.bgtq_evict(L.plan, src, dev(scores), lens32([0, 50]), 50, 16, 0, 4, dst, ds, dl, kept, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == bg.STATUS_PAGE_RANGE


def test_bounded_run_captured_and_on_another_stream():
    """A prompt, its scores, a cut to a budget, scored steps on the cut cache, windowed steps: eagerly, and the
    steps captured into a graph on another stream and replayed."""
    T, budget, steps, H, G = 400, 130, 6, 2, 4
    L = Layer(21, H, G, 384, 3, [T + steps])
    q, k, v = (x[:, :, :T].copy() for x in prompt(L))
    full, cut = L.cache(T), L.cache(160, page=16)
    out = torch.empty(q.shape, dtype=torch.float16, device="cuda")
    lse = torch.empty(q.shape[:3], device="cuda")
    scores = torch.zeros((1, H, T), device="cuda")
    bg.bgtq_prefill_window_attn(L.plan, dev(q), dev(k), dev(v), full, 0, T, out, lse=lse)
    n = bg.bgtq_prefill_score_workspace(L.plan, 1, T, T - 32)
    bg.bgtq_prefill_score(L.plan, dev(q), dev(k), lse, scores, zeros_ws(n), row0=T - 32)
    kept_scores = torch.zeros((1, H, 160), device="cuda")
    lens = lens32([0])
    kept = torch.empty((1, H, budget), dtype=torch.int32, device="cuda")
    bg.bgtq_evict(L.plan, full, scores, lens32([T]), T, budget, 4, 16, cut, kept_scores, lens, kept)
    torch.cuda.synchronize()
    assert lens.tolist() == [budget]
    # the oracle's run: keys and values kept per head, then one more token a step
    keys = [[L.enc[0][h]["khat"][j] for j in kept[0, h].tolist()] for h in range(H)]
    vals = [[L.enc[0][h]["vhat"][j] for j in kept[0, h].tolist()] for h in range(H)]
    weight = [np.concatenate([kept_scores[0, h, :budget].double().cpu().numpy(), np.zeros(30)]) for h in range(H)]

    qd = dev(L.q)
    kn, vn = torch.empty((1, H, 128), dtype=torch.float16, device="cuda"), torch.empty((1, H, 128), dtype=torch.float16, device="cuda")
    pos, now = lens32([0]), lens32([0])
    o1, o2 = torch.empty((1, H * G, 128), device="cuda"), torch.empty((1, H * G, 128), device="cuda")
    ws1 = zeros_ws(bg.bgtq_decode_score_workspace(L.plan, 1, 160))
    ws2 = zeros_ws(bg.bgtq_decode_window_workspace(L.plan, 1, 160, 4, 50))

    def step():
        bg.bgtq_decode_score_attn(L.plan, qd, cut, now, 160, kept_scores, kept_scores, o1, ws1, k_new=kn, v_new=vn, pos_new=pos)
        bg.bgtq_decode_window_attn(L.plan, qd, cut, now, 160, 4, 50, o2, ws2)

    def feed(i):
        kn.copy_(dev(L.li[0].k[None, :, T + i]))
        vn.copy_(dev(L.li[0].v[None, :, T + i]))
        pos.fill_(budget + i)
        now.fill_(budget + i + 1)

    def check(i):
        for h in range(H):
            keys[h].append(L.enc[0][h]["khat"][T + i])
            vals[h].append(L.enc[0][h]["vhat"][T + i])
            K, V = np.array(keys[h], np.float64), np.array(vals[h], np.float64)
            w = O.attention_weights(L.q[0, h * G:(h + 1) * G], K)
            m = len(K)
            weight[h][m - 1] = 0
            weight[h][:m] += w.sum(0)
            d = L.logit_error(0, h, np.arange(T + steps))
            tol = np.expm1(2 * d) + 2.0 ** -15
            got = kept_scores[0, h, :m].double().cpu().numpy()
            assert (np.abs(got - weight[h][:m]) <= tol * (i + 1) * G + 2.0 ** -20 * weight[h][:m]).all()
            rows = slice(h * G, (h + 1) * G)
            cancel = 2.0 ** -20 * np.linalg.norm(V, axis=1).max()  # as in check_decode_out
            assert (np.abs(o1[0, rows].double().cpu().numpy() - w @ V) <= tol * (w @ np.abs(V)) + cancel).all()
            at = O.decode_visible(m, 4, 50)
            w2 = O.attention_weights(L.q[0, rows], K[at])
            assert (np.abs(o2[0, rows].double().cpu().numpy() - w2 @ V[at]) <= tol * (w2 @ np.abs(V[at])) + cancel).all()

    feed(0)
    step()
    torch.cuda.synchronize()
    check(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        feed(1)
        step()
    torch.cuda.synchronize()
    check(1)
    with torch.cuda.graph(g, stream=side):
        step()
    for i in range(2, steps):
        feed(i)
        g.replay()
        torch.cuda.synchronize()
        check(i)


@pytest.mark.parametrize("T", [100, 129])
def test_prompt_calls_keep_what_is_not_finite_to_its_own_head(T):
    """A head of NaN and infinities: the heads before it, whose last tiles end inside it, are as without it."""
    L = Layer(31, 2, 2, 384, 3, [T, T])
    q, k, v = prompt(L)
    res = []
    for bad in (False, True):
        if bad:
            q[1], k[1], v[1] = np.nan, np.inf, np.nan
            q[1, 0], k[1, 0], v[1, 0] = np.inf, np.nan, -np.inf
        out = torch.zeros(q.shape, dtype=torch.float32, device="cuda")
        lse = torch.zeros(q.shape[:3], device="cuda")
        bg.bgtq_prefill_window_attn(L.plan, dev(q), dev(k), dev(v), L.cache(T + T % 2), 3, 40, out, lse=lse)
        got = [out[0].clone(), lse[0].clone()]
        for row0 in (0, T - 9):
            scores = torch.zeros((2, 2, T), device="cuda")
            n = bg.bgtq_prefill_score_workspace(L.plan, 2, T, row0)
            bg.bgtq_prefill_score(L.plan, dev(q), dev(k), lse, scores, zeros_ws(n), row0=row0, sinks=3, window=40)
            got.append(scores[0].clone())
        res.append(got)
    torch.cuda.synchronize()
    for a, b in zip(*res):
        assert torch.isfinite(b).all() and torch.equal(a, b)


def test_evicted_lengths_go_straight_into_decode():
    """dst_lens as the next call's seq_lens, with nothing in between: a decode reads its lengths before it waits."""
    L = Layer(32, 2, 4, 384, 3, [900, 700, 60])
    cap = 900
    cache = L.cache(cap)
    L.fill(cache)
    scores = dev(score_kinds("spread", (3, 2, cap), 3))
    q = dev(L.q)
    for keep in (300, 40, 64, 500, 33):
        dst = L.cache(keep + keep % 2)
        ds = torch.zeros((3, 2, dst.capacity), device="cuda")
        kept = torch.zeros((3, 2, keep), dtype=torch.int32, device="cuda")
        lens = lens32([0, 0, 0])
        ws = zeros_ws(bg.bgtq_decode_window_workspace(L.plan, 3, keep, 2, 20))
        ws2 = zeros_ws(bg.bgtq_decode_score_workspace(L.plan, 3, keep))
        out = [torch.zeros((3, 8, 128), device="cuda") for _ in range(4)]
        src_lens = lens32(L.lens)
        torch.cuda.synchronize()
        bg.bgtq_evict(L.plan, cache, scores, src_lens, cap, keep, 2, 5, dst, ds, lens, kept)
        bg.bgtq_decode_window_attn(L.plan, q, dst, lens, keep, 2, 20, out[0], ws)
        bg.bgtq_evict(L.plan, cache, scores, src_lens, cap, keep, 2, 5, dst, ds, lens, kept)
        bg.bgtq_decode_score_attn(L.plan, q, dst, lens, keep, ds, ds, out[1], ws2)
        torch.cuda.synchronize()
        assert lens.tolist() == [min(n, keep) for n in L.lens]
        bg.bgtq_decode_window_attn(L.plan, q, dst, lens, keep, 2, 20, out[2], ws)
        torch.cuda.synchronize()
        bg.bgtq_decode_score_attn(L.plan, q, dst, lens, keep, ds, ds, out[3], ws2)
        torch.cuda.synchronize()
        assert torch.equal(out[0], out[2]) and torch.equal(out[1], out[3])


@pytest.mark.parametrize("page", [0, 16])
def test_norms_that_are_not_finite_stay_out_of_the_windows_last_tiles(page):
    """Records next to the sinks and next to the window, in the tiles that hold both kinds, with norms of NaN and infinity."""
    L = Layer(33, 2, 4, 384, 3, [300])
    cache = L.cache(304, page)
    L.fill(cache)
    want = window_call(L, cache, 5, 50)
    table = cache.page_table[0].tolist() if page else None
    for pos in (5, 9, 15, 240, 249):  # (the window starts at 250, its tile at 240)
        for h in range(2):
            at = (table[pos // page] * 2 + h) * page + pos % page if page else h * 304 + pos
            cache.k_norm[at] = float("nan")
            cache.v_norm[at] = float("inf") if pos & 1 else float("nan")
    got = window_call(L, cache, 5, 50)
    torch.cuda.synchronize()
    assert torch.isfinite(got).all() and torch.equal(got, want)
    assert torch.isnan(window_call(L, cache, 6, 50)).any()  # (position 5 seen)


@pytest.mark.parametrize("row0", [0, 290])
def test_prompt_scores_of_a_log_sum_exp_out_of_range(row0):
    L = Layer(34, 1, 2, 384, 3, [300])
    q, k, _ = prompt(L)
    lse = torch.full((1, 2, 300), 1.4e6, device="cuda")  # 1.58e7 / 128^-0.5: weights of 0
    n = bg.bgtq_prefill_score_workspace(L.plan, 1, 300, row0)
    for bad in (None, 2e6, -2e6):
        scores = torch.full((1, 1, 300), GARBAGE, device="cuda")
        if bad is not None:
            lse[0, 1, 295] = bad
        bg.bgtq_prefill_score(L.plan, dev(q), dev(k), lse, scores, zeros_ws(n), row0=row0)
        torch.cuda.synchronize()
        seen = scores[0, 0].cpu()
        assert torch.isnan(seen[:296]).all() if bad else (seen[:296] == 0).all()
        assert (seen[296:] == 0).all()


def test_a_workspace_serves_every_shorter_length_on_this_gpu():
    L = Layer(35, 2, 4, 384, 3, [400, 90, 7])
    for batch in (1, 3, 20, 37, 160):
        last = [0, 0]
        for n in range(1, 40000, 53):
            now = [bg.bgtq_decode_window_workspace(L.plan, batch, n, 0, 1 << 40), bg.bgtq_decode_score_workspace(L.plan, batch, n)]
            assert now[0] >= last[0] and now[1] >= last[1], (batch, n)
            last = now
    # one workspace over calls of growing and shrinking lengths
    cache = L.cache(400)
    L.fill(cache)
    ws = zeros_ws(bg.bgtq_decode_score_workspace(L.plan, 3, 400))
    s = torch.zeros((3, 2, 400), device="cuda")
    for n in (7, 400, 33, 129, 400, 1):
        M = Layer.__new__(Layer)
        M.__dict__.update(L.__dict__, lens=[min(n, x) for x in L.lens])
        out = score_call(M, cache, s, s, ws=ws)
        win = window_call(M, cache, 4, 60, ws=ws)
        torch.cuda.synchronize()
        check_decode_out(M, out.double().cpu().numpy(), np.arange, False)
        check_decode_out(M, win.double().cpu().numpy(), lambda x: O.decode_visible(x, 4, 60), False)


def test_tensors_of_the_host_are_refused():
    L = Layer(36, 1, 2, 384, 3, [20])
    cache = L.cache(20)
    L.fill(cache)
    host = torch.zeros(1 << 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="workspace"):
        window_call(L, cache, 4, 8, ws=host)
    with pytest.raises(ValueError, match="status"):
        window_call(L, cache, 4, 8, status=torch.zeros(1, dtype=torch.int32))
    s = torch.zeros((1, 1, 20), device="cuda")
    with pytest.raises(ValueError, match="workspace"):
        score_call(L, cache, s, s, ws=host)
    with pytest.raises(ValueError, match="scores_out must be a CUDA"):
        score_call(L, cache, s, s.cpu())
    torch.cuda.synchronize()


def test_prefill_window_into_a_paged_cache_with_a_recent_key_buffer():
    T = 300
    L = Layer(37, 2, 3, 384, 3, [T, T])
    q, k, v = prompt(L)
    pair = []
    for call in (lambda c, o, st: bg.bgtq_prefill_window_attn(L.plan, dev(q), dev(k), dev(v), c, 0, T, o, status=st),
                 lambda c, o, st: bg.bgtq_prefill_attn(L.plan, dev(q), dev(k), dev(v), c, o, status=st)):
        c, o, st = L.cache(304, page=16, recent=20), torch.empty(q.shape, device="cuda"), lens32([0])
        c.page_table[1, 3] = -1  # (its records are nowhere)
        call(c, o, st)
        torch.cuda.synchronize()
        assert int(st.item()) == bg.STATUS_PAGE_RANGE
        pair.append((c, o))
    (a, oa), (b, ob) = pair
    for n in ("k_codes", "v_codes", "k_norm", "v_norm", "k_recent"):
        assert torch.equal(getattr(a, n), getattr(b, n)), n
    # fp16 probabilities on both sides: 2^-11 sum w |v| each, at most 2^-10 max |v|; as much again for the sums
    assert (oa - ob).abs().max().item() < 2.0 ** -9 * np.abs(v.astype(np.float32)).max()


def test_prompt_calls_captured_and_on_two_streams():
    """Prefill, scores and the cut of a layer in one graph, replayed on new inputs; the scores of two layers at once."""
    T, keep = 700, 90
    layers = [Layer(38 + i, 2, 4, 384, 3, [T]) for i in range(2)]
    P = [prompt(L) for L in layers]
    plan = layers[0].plan
    n = bg.bgtq_prefill_score_workspace(plan, 1, T, 0)
    assert n > 0

    class Run:
        def __init__(self, L):
            self.q, self.k, self.v = (torch.zeros(x.shape, dtype=torch.float16, device="cuda") for x in P[0])
            self.full, self.cut = bg.Cache(plan, 1, T), bg.Cache(plan, 1, keep)
            self.out = torch.empty(self.q.shape, dtype=torch.float16, device="cuda")
            self.lse = torch.empty(self.q.shape[:3], device="cuda")
            self.scores, self.kept_scores = torch.empty((1, 2, T), device="cuda"), torch.empty((1, 2, keep), device="cuda")
            self.kept, self.lens = torch.empty((1, 2, keep), dtype=torch.int32, device="cuda"), lens32([0])
            self.src, self.ws = lens32([T]), zeros_ws(n)
            self.feed(L)

        def feed(self, i):
            for x, y in zip((self.q, self.k, self.v), P[i]):
                x.copy_(dev(y))

        def go(self):
            bg.bgtq_prefill_window_attn(plan, self.q, self.k, self.v, self.full, 3, 200, self.out, lse=self.lse)
            bg.bgtq_prefill_score(plan, self.q, self.k, self.lse, self.scores, self.ws, sinks=3, window=200)
            bg.bgtq_evict(plan, self.full, self.scores, self.src, T, keep, 3, 20, self.cut, self.kept_scores, self.lens, self.kept)

        def results(self):
            return [x.clone() for x in (self.out, self.lse, self.scores, self.kept_scores, self.kept, self.lens,
                                        self.cut.k_codes, self.cut.v_codes, self.cut.k_norm, self.cut.v_norm)]

    def equal(a, b):
        return all(torch.equal(x, y) for x, y in zip(a, b))

    want = []
    for i in range(2):
        r = Run(i)
        torch.cuda.synchronize()
        r.go()
        torch.cuda.synchronize()
        want.append(r.results())
    assert not equal(*want)
    # one graph, captured on another stream
    r, side, g = Run(0), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        r.go()
    for i in (0, 1, 0):
        r.feed(i)
        for x in (r.scores, r.kept_scores, r.out, r.lse):
            x.fill_(GARBAGE)
        g.replay()
        torch.cuda.synchronize()
        assert equal(r.results(), want[i])
    # two layers at once
    runs, streams = [Run(0), Run(1)], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for x, s in zip(runs, streams):
            with torch.cuda.stream(s):
                x.go()
    torch.cuda.synchronize()
    assert equal(runs[0].results(), want[0]) and equal(runs[1].results(), want[1])
