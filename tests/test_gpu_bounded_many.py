"""GPU: the bounded-cache calls with more work than one wave of CTAs: batches
whose decode splits have no clusters, prompt scores with several items or key
tiles per CTA, evictions of every selection instance; and softmax scales other
than the usual one.  Tolerances as in test_gpu_bounded.py (the prompt scores'
reference is computed in float64 on the GPU)."""

import numpy as np
import pytest

import rope_aware_quantized_gb300 as bg
from oracle import bgtq_oracle as O

from tests.test_gpu_bounded import (GARBAGE, SCALE, Layer, bare_layer, gather, lens32, prompt, random_cache, score_kinds,
                                    zeros_ws)
from tests.test_gpu_parity import dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


# ----------------------------------------------------------------------------- decode


class Wide(Layer):
    """A batch over a few distinct sequences (sequence b's tokens are a prefix of those of b mod `distinct`)."""

    def __init__(self, seed, H, G, bpk, bv, lens, distinct):
        super().__init__(seed, H, G, bpk, bv, [max(lens)] * distinct)
        pick = [b % distinct for b in range(len(lens))]
        self.lens = list(lens)
        self.li, self.enc = [self.li[i] for i in pick], [self.enc[i] for i in pick]
        self.q = np.stack([np.roll(self.q[i], b // distinct, axis=0) for b, i in enumerate(pick)])


def new_token(L):
    at = [max(n - 1, 0) for n in L.lens]
    B = range(len(L.lens))
    return dict(k_new=dev(np.stack([L.li[b].k[:, at[b]] for b in B])), v_new=dev(np.stack([L.li[b].v[:, at[b]] for b in B])),
                pos_new=lens32(at))


def check_out(L, got, visible, half, scale=SCALE):
    """out [B][H*G][128] against the oracle's attention over each sequence's visible positions."""
    for b, n in enumerate(L.lens):
        at = visible(n)
        for h in range(L.H):
            rows = slice(h * L.G, (h + 1) * L.G)
            if n == 0:
                assert (got[b, rows] == 0).all()
                continue
            e = L.enc[b][h]
            w = O.attention_weights(L.q[b, rows], e["khat"][at], scale)
            v = e["vhat"][at].astype(np.float64)
            want, d = w @ v, logit_error(L, b, h) * scale / SCALE
            tol = (np.expm1(2 * d) + 2.0 ** -16) * (w @ np.abs(v)) + 2.0 ** -20 * np.linalg.norm(v, axis=1).max()
            if half:
                tol = tol + 2.0 ** -11 * np.abs(want) + 2.0 ** -25
            assert (np.abs(got[b, rows] - want) <= tol).all(), (b, h, np.abs(got[b, rows] - want).max(), tol.min())


def logit_error(L, b, h):
    n = L.lens[b]
    M = Layer.__new__(Layer)  # (the sequence's own tokens alone)
    e = {k: v[:n] if k in ("kcodes", "krho") else v for k, v in L.enc[b][h].items()}
    li = type("T", (), {"k": L.li[b].k[:, :n]})
    M.__dict__.update(L.__dict__, enc={b: {h: e}}, li={b: li})
    return M.logit_error(b, h, np.arange(n))


def check_scores(L, got, before, rest, step, scale=SCALE):
    for b, n in enumerate(L.lens):
        for h in range(L.H):
            behind = rest[b, h, n:].copy()
            if step and n == 0:
                behind[0] = 0  # (the new token's position, not attended)
            assert np.array_equal(got[b, h, n:], behind)  # behind the sequence: as they were
            if n == 0:
                continue
            w = O.attention_weights(L.q[b, h * L.G:(h + 1) * L.G], L.enc[b][h]["khat"][:n], scale).sum(0)
            was = before[b, h, :n].astype(np.float64)
            if step:
                was[n - 1] = 0
            # (a head's weight below the normal range, 2^-126, may be flushed to 0: by the exponential, or
            # by the product with 1 / L <= 1, at most 2^-126 each time)
            tol = (np.expm1(2 * logit_error(L, b, h) * scale / SCALE) + 2.0 ** -17) * w + 2.0 ** -23 * np.abs(was + w)
            tol = tol + L.G * 2.0 ** -125
            assert (np.abs(got[b, h, :n] - (was + w)) <= tol).all(), (b, h)


def ragged(B, longest, seed, first=()):
    r = np.random.default_rng(seed)
    return [*first, *(int(x) for x in r.integers(0, longest + 1, B - len(first)))]


def decode_case(L, cap, page, step, half, sinks, window, scale=SCALE):
    """The windowed and the scoring step over one batch, twice on one workspace each."""
    B, max_len = len(L.lens), max(L.lens)
    cache = L.cache(cap, page)
    L.fill(cache, [max(n - 1, 0) for n in L.lens] if step else None)
    new = new_token(L) if step else {}
    q, lens, dt = dev(L.q), lens32(L.lens), torch.float16 if half else torch.float32
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = zeros_ws(bg.bgtq_decode_window_workspace(L.plan, B, max_len, sinks, window))
    outs = [torch.full((B, L.H * L.G, 128), GARBAGE, dtype=dt, device="cuda") for _ in range(4)]
    for out in outs[:2]:
        bg.bgtq_decode_window_attn(L.plan, q, cache, lens, max_len, sinks, window, out, ws, softmax_scale=scale, status=st, **new)
    ws = zeros_ws(bg.bgtq_decode_score_workspace(L.plan, B, max_len))
    before = np.random.default_rng(1).random((B, L.H, cap)).astype(np.float32)
    two, one = torch.full(before.shape, GARBAGE, device="cuda"), dev(before)
    bg.bgtq_decode_score_attn(L.plan, q, cache, lens, max_len, dev(before), two, outs[2], ws, softmax_scale=scale, status=st, **new)
    bg.bgtq_decode_score_attn(L.plan, q, cache, lens, max_len, one, one, outs[3], ws, softmax_scale=scale, status=st, **new)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[2], outs[3])  # (the counters were left at 0)
    check_out(L, outs[0].double().cpu().numpy(), lambda n: O.decode_visible(n, sinks, window), half, scale)
    check_out(L, outs[2].double().cpu().numpy(), np.arange, half, scale)
    check_scores(L, two.cpu().numpy(), before, np.full_like(before, GARBAGE), step, scale)
    check_scores(L, one.cpu().numpy(), before, before, step, scale)


@pytest.mark.parametrize("B,H,G,bits,page,step,half", [
    (24, 2, 7, (384, 3), 0, False, False),
    (24, 2, 8, (256, 2), 16, True, True),
    (41, 1, 1, (128, 4), 0, True, False),
])
def test_splits_without_clusters(B, H, G, bits, page, step, half):
    """More units than clusters of 8 splits fit the GPU: several one-CTA splits a unit, all query heads merged by each."""
    assert B * H * 8 > 2 * sms()
    L = Wide(41, H, G, bits[0], bits[1], ragged(B, 700, B, (700, 0, 1, 16, 17, 699, 305)), 3)
    decode_case(L, 704, page, step, half, 5, 300)


@pytest.mark.parametrize("page,step", [(0, True), (64, False)])
def test_one_split_of_more_than_4096_tokens(page, step):
    """A unit per CTA, and a sequence of 6000 tokens (5520 of them in the window) in a single split."""
    B = (2 * sms() - 16) // 2  # two units a sequence: one wave
    L = Wide(42, 2, 2, 384, 3, ragged(B, 40, 3, (37, 6000)), 2)
    assert max(O.decode_visible(6000, 20, 5500).shape) > 4096
    decode_case(L, 6016, page, step, False, 20, 5500)


@pytest.mark.parametrize("scale", [0.11, 0.02])
def test_decode_softmax_scale(scale):
    decode_case(Wide(43, 2, 3, 384, 3, [300, 0, 33, 129], 2), 304, 0, True, False, 4, 50, scale)


# ----------------------------------------------------------------------------- prompts


def prompt_reference(q, k, row0, sinks, window, scale):
    """One KV head in float64: q [G][T][128], k [T][128] -> (lse [G][T - row0], score [T], bound of a logit's error)."""
    T = k.shape[0]
    qd, kd = q[:, row0:].double(), k.double()
    s = (qd @ kd.T) * scale
    i, j = torch.arange(row0, T, device="cuda")[:, None], torch.arange(T, device="cuda")[None, :]
    s.masked_fill_(~((j <= i) & ((j < sinks) | (j > i - window))), float("-inf"))
    lse = torch.logsumexp(s, 2)
    mag = (qd.abs() @ kd.abs().T).max().item() if row0 < T else 0.0
    return lse, torch.exp(s - lse[..., None]).sum((0, 1)), scale * 2.0 ** -17 * mag


def prompt_plan(H, G):
    return bg.bgtq_plan_create(np.full((H, 64), 3, np.uint8), np.ones((H, 64)), G, 384, 3, 1)


def prompt_inputs(B, H, G, T, seed):
    """q, k of a few units' logits, different in every head."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (1.5 * torch.randn((B, H * G, T, 128), device="cuda", generator=g)).half(), torch.randn((B, H, T, 128), device="cuda",
                                                                                                  generator=g).half()


def score_case(B, H, G, T, row0, sinks, window, scale=SCALE):
    plan = prompt_plan(H, G)
    q, k = prompt_inputs(B, H, G, T, T + G)
    lse = torch.full((B, H * G, T), float("nan"), device="cuda")  # rows before row0 are not read
    want, tol = torch.zeros((B, H, T), dtype=torch.float64, device="cuda"), torch.zeros((B, H, T), dtype=torch.float64, device="cuda")
    for b in range(B):
        for h in range(H):
            rows = slice(h * G, (h + 1) * G)
            x, w, d = prompt_reference(q[b, rows], k[b, h], row0, sinks, window, scale)
            lse[b, rows, row0:] = x.float()
            want[b, h] = w
            d += 2.0 ** -22 * x.abs().max().item()  # lse and its product with log2 e in fp32
            tol[b, h] = (np.expm1(2 * d) + 2.0 ** -17) * w + 1e-30
    n = bg.bgtq_prefill_score_workspace(plan, B, T, row0)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = [torch.full((B, H, T + 1), GARBAGE, device="cuda") for _ in range(3)]
    for x in got:
        bg.bgtq_prefill_score(plan, q, k, lse, x, ws, row0=row0, sinks=sinks, window=window, softmax_scale=scale, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and (got[0][..., T] == GARBAGE).all()
    off = (got[0][..., :T].double() - want).abs()
    assert (off <= tol).all(), (off - tol).max().item()
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])  # the same bits on every run
    return n // (4 * B * H * T) or 1


@pytest.mark.parametrize("B,H,G,T,row0,sinks,window", [
    (8, 4, 2, 1500, 0, 0, 1500),        # items of 12, 10, 8 .. row tiles, two parts
    (8, 4, 2, 1500, 900, 5, 200),       # items without row tiles between others (keys 256 .. 511)
    (10, 2, 3, 1300, 37, 4, 700),       # odd numbers of row tiles
    (16, 10, 1, 700, 0, 0, 700),        # one part
    (10, 4, 8, 2000, 1950, 3, 1000),    # two query heads' rows in a tile
])
def test_prompt_scores_with_several_items_per_cta(B, H, G, T, row0, sinks, window):
    parts = score_case(B, H, G, T, row0, sinks, window)
    assert B * H * parts * -(-T // 256) > 2 * sms()


@pytest.mark.parametrize("G,rows,sinks,window", [
    (4, 40, 0, 2500),      # 256 columns
    (4, 40, 5, 300),       # tiles that no row sees, between the sinks' and the window's
    (4, 20, 3, 1500),      # 128 columns
    (1, 200, 0, 1100),     # the rows of one query head
    (8, 1, 130, 1),        # one row
])
def test_prompt_scores_with_several_key_tiles_per_cta(G, rows, sinks, window):
    B, H, T = 16, 4, 2500  # 64 x 20 key tiles
    assert B * H * 20 > 4 * sms()
    score_case(B, H, G, T, T - rows, sinks, window)


@pytest.mark.parametrize("scale", [0.2, 0.011])
@pytest.mark.parametrize("row0", [0, 580])
def test_prompt_score_softmax_scale(row0, scale):
    score_case(2, 2, 3, 600, row0, 4, 100, scale)


@pytest.mark.parametrize("scale", [0.2, 0.011])
@pytest.mark.parametrize("half", [False, True])
def test_prefill_window_softmax_scale(half, scale):
    T, H, G = 450, 2, 3
    L = Layer(44, H, G, 384, 3, [T])
    q, k, v = prompt(L)
    out = torch.full(q.shape, GARBAGE, dtype=torch.float16 if half else torch.float32, device="cuda")
    lse = torch.full(q.shape[:3], GARBAGE, device="cuda")
    bg.bgtq_prefill_window_attn(L.plan, dev(q), dev(k), dev(v), L.cache(T), 5, 70, out, lse=lse, softmax_scale=scale)
    torch.cuda.synchronize()
    for h in range(H):
        rows = slice(h * G, (h + 1) * G)
        want, wlse, w = O.prefill_window(q[0, rows], k[0, h], v[0, h], 5, 70, scale)
        kd, va = np.abs(k[0, h].astype(np.float64)), np.abs(v[0, h].astype(np.float64))
        d = scale * 2.0 ** -17 * max((np.abs(q[0, i].astype(np.float64)) @ kd.T).max() for i in range(rows.start, rows.stop))
        tol = (2.0 ** -11 + np.expm1(2 * d) + 2.0 ** -16) * np.einsum("gij,jd->gid", w, va) + T * 2.0 ** -25 * va.max()
        if half:
            tol = tol + 2.0 ** -11 * np.abs(want) + 2.0 ** -25
        assert (np.abs(out[0, rows].double().cpu().numpy() - want) <= tol).all()
        dl = np.abs(lse[0, rows].double().cpu().numpy() - wlse)
        assert (dl <= d + 2.0 ** -17 + 2.0 ** -21 * np.abs(wlse)).all(), dl.max()


@pytest.mark.parametrize("half", [False, True])
def test_prefill_window_of_many_blocks(half):
    """More CTAs than SMs, blocks with tiles of all kinds; the same bits on every run."""
    B, H, G, T, sinks, window = 3, 2, 8, 1531, 5, 255
    assert B * H * (G // 2) * -(-T // 128) > sms()
    plan = prompt_plan(H, G)
    q, k = prompt_inputs(B, H, G, T, 9)
    v = torch.randn(k.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(10)).half()
    runs = []
    for _ in range(4):
        out = torch.full(q.shape, GARBAGE, dtype=torch.float16 if half else torch.float32, device="cuda")
        lse = torch.full(q.shape[:3], GARBAGE, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        bg.bgtq_prefill_window_attn(plan, q, k, v, bg.Cache(plan, B, T + 1), sinks, window, out, lse=lse, status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        runs.append((out, lse))
    for out, lse in runs[1:]:
        assert torch.equal(out, runs[0][0]) and torch.equal(lse, runs[0][1])
    out, lse = runs[0]
    i, j = torch.arange(T, device="cuda")[:, None], torch.arange(T, device="cuda")[None, :]
    hidden = ~((j <= i) & ((j < sinks) | (j > i - window)))
    for b in range(B):
        for h in range(H):
            rows = slice(h * G, (h + 1) * G)
            qd, kd, vd = q[b, rows].double(), k[b, h].double(), v[b, h].double()
            s = ((qd @ kd.T) * SCALE).masked_fill(hidden, float("-inf"))
            wlse, w = torch.logsumexp(s, 2), torch.softmax(s, 2)
            d = SCALE * 2.0 ** -17 * (qd.abs() @ kd.abs().T).max().item()
            want = w @ vd
            tol = (2.0 ** -11 + np.expm1(2 * d) + 2.0 ** -16) * (w @ vd.abs()) + T * 2.0 ** -25 * vd.abs().max()
            if half:
                tol = tol + 2.0 ** -11 * want.abs() + 2.0 ** -25
            assert ((out[b, rows].double() - want).abs() <= tol).all()
            assert ((lse[b, rows].double() - wlse).abs() <= d + 2.0 ** -17 + 2.0 ** -21 * wlse.abs()).all()


# ----------------------------------------------------------------------------- eviction


@pytest.mark.parametrize("B,longest,page,keep,sinks,recent,bits,kind", [
    (80, 4097, 0, 700, 4, 64, (128, 1), "few"),         # 16 keys a thread, one CTA a unit
    (80, 8192, 16, 1024, 4, 32, (128, 2), "odd"),       # the longest of them
    (80, 8193, 0, 2100, 0, 1, (256, 3), "odd"),         # 32 keys a thread
    (80, 16384, 64, 4095, 16, 100, (128, 1), "few"),    # the longest of them
    (80, 16385, 0, 333, 1, 0, (128, 1), "equal"),       # and clusters of two
    (10, 20001, 0, 5000, 4, 64, (128, 3), "odd"),       # clusters of eight, 8 keys a thread
    (10, 40001, 0, 9999, 4, 64, (128, 1), "few"),       # clusters of eight, 16 keys a thread
])
def test_evict_instances(B, longest, page, keep, sinks, recent, bits, kind):
    H = 2
    lens = ragged(B, longest, keep, (longest, 0, keep, keep + 1, longest - 1))
    plan = bare_layer(H, *bits).plan
    cap = -(-longest // max(page, 2)) * max(page, 2)
    src = random_cache(plan, H, B, cap, page, bits, 3)
    dcap = -(-keep // max(page, 2)) * max(page, 2)
    dst = random_cache(plan, H, B, dcap, page, bits, 4)
    some = (0, 1, 2, 3, B - 1)
    before = {b: gather(dst, b, H, dcap) for b in some}
    scores = score_kinds(kind, (B, H, cap), 5)
    ds, dl = torch.full((B, H, dcap), GARBAGE, device="cuda"), lens32([-7] * B)
    kept = torch.full((B, H, keep), -9, dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    bg.bgtq_evict(plan, src, dev(scores), lens32(lens), longest, keep, sinks, recent, dst, ds, dl, kept, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and dl.tolist() == [min(n, keep) for n in lens]
    k, x = kept.cpu().numpy(), ds.cpu().numpy()
    for b, n in enumerate(lens):
        for h in range(H):
            at = stay(scores[b, h], n, keep, sinks, recent)
            m = len(at)
            assert np.array_equal(k[b, h, :m], at) and (k[b, h, m:] == -1).all(), (b, h, n)
            assert np.array_equal(x[b, h, :m], scores[b, h][at], equal_nan=True) and (x[b, h, m:] == GARBAGE).all()
    for b in some:
        after, records = gather(dst, b, H, dcap), gather(src, b, H, lens[b])
        for h in range(H):
            at = stay(scores[b, h], lens[b], keep, sinks, recent)
            for got, want, old in zip(after[h], records[h], before[b][h]):
                assert np.array_equal(got[:len(at)], want[at]) and np.array_equal(got[len(at):], old[len(at):])


def stay(scores, n, keep, sinks, recent):
    """O.evict_positions by one stable sort (a batch of long sequences)."""
    if n <= keep:
        return np.arange(n)
    x = scores[sinks:n - recent].astype(np.float64)
    order = np.lexsort((np.arange(len(x)), -np.where(np.isnan(x), 0.0, x), np.isnan(x)))
    mid = sinks + order[:keep - sinks - recent]
    return np.sort(np.concatenate([np.arange(sinks), mid, np.arange(n - recent, n)])).astype(np.int64)


def test_the_sorted_reference_is_the_oracles():
    for kind in ("few", "odd", "equal", "spread"):
        x = score_kinds(kind, (300,), 8)
        for n, keep, sinks, recent in ((300, 50, 4, 7), (299, 1, 0, 0), (40, 40, 3, 3), (77, 12, 5, 7)):
            assert np.array_equal(stay(x, n, keep, sinks, recent), O.evict_positions(x, n, keep, sinks, recent))
