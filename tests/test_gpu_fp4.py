"""GPU: the 4-bit cache: appended bytes, attention over them, and both together.

Tolerances (derived, not fitted).  Bytes are equal to the oracle's.  A cached
key or value is exact in fp16, and a product of two fp16 numbers in fp32; a
logit sums 128 of them in fp32 (128 half steps, 2^-17 of the sum of their
magnitudes) and is scaled by two rounded factors: off by d = 2^-17 + 2^-22 of
scale |q| |k|.  A weight is then off by expm1(2 d) and the exponential's
2^-21 of itself; its two fp16 parts by 2^-22, or 2^-33 of the row's largest
weight, whichever is more (the parts' smallest step is 2^-24, half of it
2^-25, and the largest weight is 2^8 or more when the reference is set); an
output's sums, in chains of
at most n / 8 + 64 steps of fp32, by 2^-24 a step (rounded towards zero by the
tensor cores: 2^-23) of sum w |v|.  For an fp16 output weights are rounded to
fp16, 2^-11 (below fp16's normal range 2^-25 of the largest, 2^-17 of a weight's
share over 256 positions), and the output adds half a step, 2^-11.
"""

import ctypes

import numpy as np
import pytest

import rope_aware_quantized_gb300 as bg
from oracle import rope_fp4_oracle as F

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

SCALE = 1 / np.sqrt(128)
INV = 1e6 ** (-np.arange(64) / 64)
MIXED = [i % 3 for i in range(64)]


@pytest.fixture(autouse=True)
def seeded():
    torch.manual_seed(20)


def i32(x):
    return torch.as_tensor(np.asarray(x, np.int32)).cuda()


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def new_cache(H, B, cap, page=0, spare=0, seed=0):
    """A cache full of random bytes (scales that are no numbers among them), its pages shuffled."""
    c = bg.Fp4Cache(H, B, cap, page_tokens=page, n_pages=B * cap // page + spare if page else 0)
    g = gen(seed)
    c.groups.copy_(torch.randint(0, 256, c.groups.shape, generator=g, device="cuda", dtype=torch.uint8))
    if page:
        c.page_table.copy_(torch.randperm(c.n_pages, generator=g, device="cuda")[:c.page_table.numel()].to(torch.int32).view_as(c.page_table))
    return c


def group_rows(c, b, h):
    """Indices of the groups of (b, h) in the pool, in position order."""
    n = np.arange(c.capacity // 16)
    if not c.page_tokens:
        return (b * c.n_kv_heads + h) * (c.capacity // 16) + n
    P = c.page_tokens // 16
    t = c.page_table.cpu().numpy().astype(np.int64)
    return (t[b][n // P] * c.n_kv_heads + h) * P + n % P


def cached(c, b, h, n):
    """Keys and values [n][128] float64 that the cache's bytes stand for."""
    g = c.groups.view(-1, F.GROUP_BYTES).cpu().numpy()[group_rows(c, b, h)[:-(-n // 16)]]
    kc, ks, vc, vs = F.read(g)
    return [F.fp4_value(x, s).reshape(-1, 128)[:n] for x, s in ((kc, ks), (vc, vs))]


def check_bytes(before, c, k, v, starts, keep=lambda b, t: True):
    """The pool after an append of rotated keys k and values v [B][H][T][128] (numpy fp16)."""
    want = before.copy().reshape(-1, F.GROUP_BYTES)
    B, H, T, _ = k.shape
    for b in range(B):
        for h in range(H):
            at = group_rows(c, b, h)
            kc, ks = F.fp4_encode(k[b, h])
            vc, vs = F.fp4_encode(v[b, h])
            for t in range(T):
                if keep(b, t):
                    p = starts[b] + t
                    F.write(want[at[p // 16]], p % 16, kc[t], ks[t], vc[t], vs[t])
    got = c.groups.cpu().numpy().reshape(-1, F.GROUP_BYTES)
    bad = np.argwhere(got != want)
    assert len(bad) == 0, (len(bad), bad[:5], [(got[tuple(i)], want[tuple(i)]) for i in bad[:5]])


def hard_rows(rng, shape):
    """Rows whose blocks have ties, zeros, negative zeros, subnormals, one big value, and the type's largest."""
    x = (rng.standard_normal(shape) * 10.0 ** rng.uniform(-6, 3, (*shape[:-1], 1))).astype(np.float16)
    x[..., 0:16] = rng.choice([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -1.25, -5], (*shape[:-1], 16))
    x[..., 16:32] = 0
    x[..., 20] = -0.0
    x[..., 32:48] = rng.choice([65504, -65504, 61440, 5120, 0], (*shape[:-1], 16))
    x[..., 48:64] = (rng.integers(0, 64, (*shape[:-1], 16)) * 2.0 ** -24).astype(np.float16)
    x[..., 64:80] = (rng.integers(-600, 600, (*shape[:-1], 16)) * 2.0 ** -24).astype(np.float16)
    x[..., 80] = 1000
    return x


@pytest.mark.parametrize("B,H,T,cap,page,starts", [
    (1, 1, 1, 16, 0, [0]), (1, 1, 1, 16, 0, [15]), (3, 2, 1, 64, 16, [0, 17, 62]), (2, 3, 2, 64, 0, [14, 15]),
    (2, 1, 16, 64, 32, [0, 16]), (2, 2, 17, 64, 0, [0, 31]), (1, 2, 100, 256, 64, [77]), (1, 1, 333, 512, 0, [5]),
])
def test_append_bytes(B, H, T, cap, page, starts):
    rng = np.random.default_rng(T + cap)
    k, v = hard_rows(rng, (B, H, T, 128)), hard_rows(rng, (B, H, T, 128))
    c = new_cache(H, B, cap, page, spare=3, seed=T)
    before = c.groups.cpu().numpy()
    st = status()
    bg.bgtq_fp4_append(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), i32(starts), c, status=st)
    check_bytes(before, c, k, v, starts)
    assert st.item() == 0


def test_every_fp16_number_in_every_place():
    """All finite fp16 numbers as a block's largest, and as the others under scales of every byte."""
    bits = np.arange(1 << 16, dtype=np.uint16)
    x = bits.view(np.float16)
    x = x[np.isfinite(x)]
    n = -(-len(x) // 128) * 128
    a = np.resize(x, n).reshape(1, 1, -1, 128)  # consecutive numbers share a block
    b = np.random.default_rng(0).permutation(np.resize(x, n)).reshape(1, 1, -1, 128)
    c = np.zeros((1, 1, len(x) // 8, 128), np.float16)
    c[..., ::16] = x[:len(x) // 8 * 8].reshape(1, 1, -1, 8)
    for k, v in ((a, b), (b, a), (c, c)):
        T = k.shape[2]
        cache = bg.Fp4Cache(1, 1, -(-T // 16) * 16)
        bg.bgtq_fp4_append(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), i32([0]), cache)
        for got, want in zip(F.read(cache.groups.cpu().numpy().reshape(-1, F.GROUP_BYTES)), (*F.fp4_encode(k[0, 0]), *F.fp4_encode(v[0, 0]))):
            assert np.array_equal(got.reshape(-1, got.shape[-1])[:T], want)


@pytest.mark.parametrize("T,layout,axis,start", [(1, 0, None, 7), (1, 1, MIXED, 8), (5, 0, MIXED, 14), (70, 1, None, 3), (70, 0, None, 0),
                                                 (129, 1, MIXED, 1), (129, 0, [0] * 16 + [1] * 24 + [2] * 24, 31)])
def test_append_rotated_equals_the_two_calls(T, layout, axis, start):
    H, B = 2, 2
    rope = bg.Rope(*bg.bgtq_rope_table(INV, 900), layout, axis)
    pos = i32(np.random.default_rng(T).integers(0, 900, (rope.axes, B, T)))
    x = torch.randn((B, T, 2 * H + 1, 128), device="cuda", generator=gen(T)).half() * 4
    k, v = x[:, :, 1:H + 1].transpose(1, 2), x[:, :, H + 1:].transpose(1, 2)
    a, b = new_cache(H, B, 256, 16, seed=1), new_cache(H, B, 256, 16, seed=1)
    bg.bgtq_fp4_append(k, v, i32([start, start + 1]), a, rope=rope, pos=pos)
    kr = torch.empty((B, H, T, 128), dtype=torch.float16, device="cuda")
    bg.bgtq_rope_rows(rope, pos, k, kr)
    bg.bgtq_fp4_append(kr, v, i32([start, start + 1]), b)
    assert torch.equal(a.groups, b.groups)
    if axis is None:
        own = i32([[start + i for i in range(T)], [start + 1 + i for i in range(T)]])
        bg.bgtq_fp4_append(k, v, i32([start, start + 1]), a, rope=rope)
        bg.bgtq_fp4_append(k, v, i32([start, start + 1]), b, rope=rope, pos=own)
        assert torch.equal(a.groups, b.groups)


def test_append_skips():
    """Past the capacity, before the start, outside the tables, onto an unmapped page: nothing else changes."""
    rng = np.random.default_rng(5)
    c = new_cache(1, 4, 64, 32, seed=2)
    c.page_table[3, 1] = -1
    before = c.groups.cpu().numpy()
    k, v = (rng.standard_normal((4, 1, 20, 128)).astype(np.float16) for _ in range(2))
    rope = bg.Rope(*bg.bgtq_rope_table(np.zeros(64), 30))  # (frequency 0: keys as they are)
    pos = np.tile(np.arange(20), (4, 1))
    pos[2, [0, 6, 7, 19]] = [30, -1, 99, 1 << 30]
    st = status()
    starts = [45, -1, 9, 25]
    bg.bgtq_fp4_append(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), i32(starts), c, rope=rope, pos=i32(pos), status=st)
    assert st.item() == bg.STATUS_APPEND_CAPACITY | bg.STATUS_ROPE_RANGE | bg.STATUS_PAGE_RANGE
    table = c.page_table.clone()
    c.page_table[3, 1] = 0  # (never written: those tokens are left out below)
    check_bytes(before, c, k, v, starts,
                lambda b, t: b >= 2 and not (b == 2 and t in (0, 6, 7, 19)) and not (b == 3 and starts[3] + t >= 32))
    c.page_table.copy_(table)


def test_more_new_tokens_than_the_capacity():
    c = new_cache(1, 2, 32, 0, seed=9)
    before = c.groups.clone()
    k = torch.randn((2, 1, 40, 128), device="cuda").half()
    st = status()
    bg.bgtq_fp4_append(k, k, i32([0, 5]), c, status=st)
    assert st.item() == bg.STATUS_APPEND_CAPACITY and torch.equal(before, c.groups)


def test_append_of_one_call_equals_many():
    """A prompt in one call (the kernel for many groups) and the same in uneven pieces."""
    H, B, T = 8, 2, 3000
    k, v = (torch.randn((B, H, T, 128), device="cuda").half() for _ in range(2))
    rope = bg.Rope(*bg.bgtq_rope_table(INV, 4000), 1, MIXED)
    pos = i32(np.random.default_rng(0).integers(0, 4000, (3, B, T)))
    a, b = new_cache(H, B, 3008, 0, seed=5), new_cache(H, B, 3008, 0, seed=5)
    bg.bgtq_fp4_append(k, v, i32([0, 8]), a, rope=rope, pos=pos)
    t = 0
    for n in (1, 15, 16, 17, 3, 100, 2000, T):
        n = min(n, T - t)
        bg.bgtq_fp4_append(k[:, :, t:t + n], v[:, :, t:t + n], i32([t, 8 + t]), b, rope=rope, pos=pos[:, :, t:t + n].contiguous())
        t += n
    assert t == T and torch.equal(a.groups, b.groups)


def test_append_skips_inside_whole_groups():
    rng = np.random.default_rng(6)
    c = new_cache(2, 1, 96, 0, seed=8)
    before = c.groups.cpu().numpy()
    k, v = (rng.standard_normal((1, 2, 70, 128)).astype(np.float16) for _ in range(2))
    rope = bg.Rope(*bg.bgtq_rope_table(np.zeros(64), 70))
    pos = np.arange(70)[None]
    bad = [10, 11, 12, 40, 61]  # a position of one group, neighbours that share bytes; cache positions 13 .. 64
    pos[0, bad] = [70, -1, 1 << 30, 71, -9]
    st = status()
    bg.bgtq_fp4_append(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), i32([3]), c, rope=rope, pos=i32(pos), status=st)
    assert st.item() == bg.STATUS_ROPE_RANGE
    check_bytes(before, c, k, v, [3], lambda b, t: t not in bad)


def test_dequant():
    c = new_cache(2, 2, 64, 16, seed=3)
    c.groups.view(-1, F.GROUP_BYTES)[:, 2048:] %= 227
    for b, h, t0, t1 in ((0, 0, 0, 64), (1, 1, 5, 23), (1, 0, 63, 64), (0, 1, 9, 9)):
        ko, vo = (torch.empty((t1 - t0, 128), device="cuda") for _ in range(2))
        bg.bgtq_fp4_dequant(c, b, h, t0, t1, ko, vo)
        k, v = cached(c, b, h, 64)
        assert np.array_equal(ko.cpu().numpy(), k[t0:t1]) and np.array_equal(vo.cpu().numpy(), v[t0:t1])


# ----------------------------------------------------------------- attention


class Case:
    """A cache with sequences of lens tokens in it, and t query rows a sequence at their end."""

    def __init__(self, H, G, t, lens, cap, page=0, seed=0, spread=1.0, contiguous=False):
        self.H, self.G, self.t, self.lens, B = H, G, t, lens, len(lens)
        self.cache = new_cache(H, B, cap, page, spare=2, seed=seed)
        g = gen(seed + 1)
        for b, n in enumerate(lens):
            if n:
                k, v = (torch.randn((1, H, n, 128), generator=g, device="cuda").half() for _ in range(2))
                one = bg.Fp4Cache.__new__(bg.Fp4Cache)
                one.__dict__.update(self.cache.__dict__)
                one.batch = 1
                one.desc = type(self.cache.desc).from_buffer_copy(self.cache.desc)
                one.address = ctypes.addressof(one.desc)
                if page:
                    one.desc.page_table += 4 * b * self.cache.max_pages
                else:
                    one.desc.groups += b * H * (cap // 16) * F.GROUP_BYTES
                bg.bgtq_fp4_append(k, v, i32([0]), one)
        if contiguous:
            self.q = torch.randn((B, H * G, t, 128), generator=g, device="cuda").half() * spread
        else:
            self.q = (torch.randn((B, t, H * G + 1, 128), generator=g, device="cuda").half() * spread)[:, :, :H * G].transpose(1, 2)
        self.seq = i32(lens)

    def run(self, half, max_len=None, ws=None, **kw):
        B, hq, t, _ = self.q.shape
        max_len = max(self.lens) if max_len is None else max_len
        out = torch.full((B, hq, t, 128), 7.25, dtype=torch.float16 if half else torch.float32, device="cuda")
        if ws is None:
            ws = torch.zeros(bg.bgtq_fp4_attn_workspace(self.H, self.G, B, t, max_len), dtype=torch.uint8, device="cuda")
        bg.bgtq_fp4_attn(self.q, self.cache, self.seq, max_len, out, ws, **kw)
        return out

    def check(self, out, half, q=None, lens=None, scale=SCALE, units=None):
        q = (self.q if q is None else q).cpu().numpy().astype(np.float64)
        got = out.double().cpu().numpy()
        assert np.isfinite(got).all()
        for b, n in enumerate(self.lens if lens is None else lens):
            for h in range(self.H):
                k, v = cached(self.cache, b, h, n) if n else (np.zeros((0, 128)),) * 2
                for a in range(h * self.G, (h + 1) * self.G):
                    if units is not None and (b, a) not in units:
                        continue
                    x = q[b, a]
                    w = F.attention(x, k, n - self.t, scale) if n else np.zeros((self.t, 0))
                    want, mag = w @ v, w @ np.abs(v)
                    kn = np.linalg.norm(k, axis=1).max() if n else 0.0
                    d = scale * np.linalg.norm(x, axis=1)[:, None] * kn * (2.0 ** -17 + 2.0 ** -22)
                    rel = np.expm1(2 * d) + 2.0 ** -21 + 2.0 ** -22 + (n / 8 + 64) * 2.0 ** -23
                    top = w.max(-1, keepdims=True, initial=0.0)
                    tol = rel * mag + 2.0 ** -33 * top * np.abs(v).sum(0)
                    if half:
                        tol = tol + 2.0 ** -11 * mag + 2.0 ** -17 * np.abs(v).max(initial=0.0)
                        tol = tol + 2.0 ** -11 * np.abs(want) + 2.0 ** -25
                    assert (np.abs(got[b, a] - want) <= tol).all(), (b, a, np.abs(got[b, a] - want).max(), tol.min())


@pytest.mark.parametrize("H,G,t,lens,cap,page", [
    (1, 1, 1, [1], 16, 0), (1, 4, 1, [0, 1, 2], 16, 0), (2, 8, 1, [15, 16, 17], 64, 16), (1, 3, 1, [255], 256, 32),
    (2, 7, 1, [129, 4096, 1000], 4096, 64), (1, 8, 1, [20000], 20480, 0), (8, 4, 1, [5, 300, 0, 77], 512, 16),
    (1, 1, 2, [1, 2, 9], 64, 0), (2, 8, 2, [0, 1, 100], 128, 16), (1, 4, 5, [3, 5, 40], 64, 0), (2, 7, 4, [1000, 2], 1024, 256),
    (1, 8, 4, [4095], 4096, 0), (1, 1, 32, [33, 31, 16], 48, 16), (3, 2, 16, [500], 512, 0),
])
@pytest.mark.parametrize("half", [False, True])
def test_attention_few_rows(H, G, t, lens, cap, page, half):
    c = Case(H, G, t, lens, cap, page, seed=cap + t, spread=1.5)
    c.check(c.run(half), half)


@pytest.mark.parametrize("H,G,t,lens,cap,page", [
    (1, 1, 33, [33, 50, 10, 0], 64, 16), (2, 8, 5, [5, 127, 128, 129], 256, 0), (1, 7, 5, [3001], 3008, 16), (2, 8, 128, [128, 300], 320, 64),
    (1, 3, 200, [199, 1000, 201], 1024, 256), (1, 8, 300, [5000], 5008, 0), (2, 1, 513, [513, 2], 528, 0), (1, 5, 77, [640], 640, 128),
])
@pytest.mark.parametrize("half", [False, True])
def test_attention_many_rows(H, G, t, lens, cap, page, half):
    c = Case(H, G, t, lens, cap, page, seed=cap + t, spread=1.5)
    c.check(c.run(half), half)


def many(B, H, G, t, top, page, seed, half, some):
    """A large ragged batch, of which the units (sequence, query head) in `some` are checked."""
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, top + 1, B)
    lens[rng.integers(0, B)] = top
    cap = -(-top // max(page, 16)) * max(page, 16)
    c = Case.__new__(Case)
    c.H, c.G, c.t, c.lens, c.seq = H, G, t, lens.tolist(), i32(lens)
    c.cache = new_cache(H, B, cap, page, spare=2, seed=seed)
    k, v = (torch.randn((B, H, cap, 128), generator=gen(seed + i), device="cuda").half() for i in (1, 2))
    bg.bgtq_fp4_append(k, v, i32(np.zeros(B)), c.cache)
    c.q = torch.randn((B, H * G, t, 128), generator=gen(seed + 3), device="cuda").half()
    out = c.run(half)
    c.check(out, half, units={(int(b), int(a)) for b, a in zip(rng.integers(0, B, some), rng.integers(0, H * G, some))})
    return c, out


@pytest.mark.parametrize("B,H,G,t,top,page", [
    (300, 2, 4, 1, 200, 16),     # more sequences than threads of a block sum up at once; several whole units a CTA
    (40, 8, 4, 1, 3000, 64),     # units that begin in one CTA's share and end in another's
    (150, 1, 8, 1, 700, 0), (20, 4, 8, 2, 900, 32), (7, 8, 5, 3, 1500, 0),
    (64, 8, 4, 5, 1100, 16), (64, 8, 8, 4, 1100, 0),  # 20 and 32 rows with work enough for one pass
    (20, 8, 1, 40, 2000, 64), (20, 8, 3, 120, 600, 16),  # more pair blocks than SMs, on the tiles
])
@pytest.mark.parametrize("half", [False, True])
def test_attention_large_batches(B, H, G, t, top, page, half):
    c, out = many(B, H, G, t, top, page, B + t, half, 40)
    assert torch.equal(out, c.run(half))  # the same bits on every run


@pytest.mark.parametrize("t", [1, 3, 40])
@pytest.mark.parametrize("layout,axis", [(0, None), (1, MIXED)])
def test_attention_rotates_the_queries(t, layout, axis):
    c = Case(2, 4, t, [300, 45, 61], 320, 16, seed=9)
    rope = bg.Rope(*bg.bgtq_rope_table(INV, 5000), layout, axis)
    pos = i32(np.random.default_rng(t).integers(0, 5000, (rope.axes, 3, t)))
    q = torch.empty(c.q.shape, dtype=torch.float16, device="cuda")
    bg.bgtq_rope_rows(rope, pos, c.q, q)
    out = c.run(False, rope=rope, pos=pos)
    c.check(out, False, q=q)
    plain = Case.run(type("C", (), dict(c.__dict__, q=q)), False)
    assert torch.equal(out, plain)  # the same bits as the two calls
    if axis is None:  # positions left out: the rows' own
        own = c.seq[:, None] - t + torch.arange(t, dtype=torch.int32, device="cuda")
        assert torch.equal(c.run(False, rope=rope), c.run(False, rope=rope, pos=own.contiguous()))


@pytest.mark.parametrize("t", [2, 50])
def test_rows_with_positions_outside_the_tables(t):
    c = Case(1, 2, t, [200, 90], 208, 0, seed=4)
    rope = bg.Rope(*bg.bgtq_rope_table(INV, 100))
    pos = np.zeros((2, t), np.int32)
    pos[0, 1], pos[1, 0] = 100, -5
    st = status()
    out = c.run(False, rope=rope, pos=i32(pos), status=st)
    assert st.item() == bg.STATUS_ROPE_RANGE
    assert (out[0, :, 1] == 0).all() and (out[1, :, 0] == 0).all()
    pos[:] = 0
    good = c.run(False, rope=rope, pos=i32(pos))
    for b, bad in ((0, 1), (1, 0)):
        keep = [i for i in range(t) if i != bad]
        assert torch.equal(out[b, :, keep], good[b, :, keep])


@pytest.mark.parametrize("t", [1, 48])
def test_lengths_outside_the_bounds(t):
    c = Case(1, 2, t, [100, 64, 0], 112, 0, seed=5)
    c.seq = i32([100, 64, -3])
    st = status()
    out = c.run(False, max_len=64, status=st)
    assert st.item() == bg.STATUS_SEQLEN_CAPACITY
    c.check(out, False, lens=[64, 64, 0])
    st.zero_()
    c.seq = i32([100, 64, 0])
    c.run(False, max_len=1 << 20, ws=torch.zeros(bg.bgtq_fp4_attn_workspace(1, 2, 3, t, 112), dtype=torch.uint8, device="cuda"), status=st)
    assert st.item() == 0


def test_an_unmapped_page_is_reported():
    c = Case(1, 4, 1, [64], 64, 16, seed=6)
    c.cache.page_table[0, 1] = c.cache.n_pages
    st = status()
    c.run(False, status=st)
    assert st.item() == bg.STATUS_PAGE_RANGE


@pytest.mark.parametrize("t", [1, 4, 64])
def test_bytes_past_the_sequence_do_not_matter(t):
    c = Case(2, 4, t, [77, 130], 256, 0, seed=7)
    a = c.run(False)
    g = c.cache.groups.view(2, 2, 16, F.GROUP_BYTES)
    raw = g.cpu().numpy().copy()
    for b, n in enumerate(c.lens):
        for h in range(2):
            for i in range(n // 16, 16):
                for p in range(max(0, n - 16 * i), 16):
                    F.write(raw[b, h, i], p, np.full(128, 15), np.full(8, 255), np.full(128, 7), np.full(8, 248))
    g.copy_(torch.from_numpy(raw))
    assert torch.equal(a, c.run(False))


@pytest.mark.parametrize("t", [1, 40])
def test_large_logits_and_one_sided_rows(t):
    """Logits of hundreds: one position takes nearly all the weight; a maximum that keeps moving up."""
    c = Case(1, 4, t, [700], 704, 0, seed=8, spread=40.0)
    c.check(c.run(False, softmax_scale=0.05), False, scale=0.05)
    n = 700
    ramp = torch.linspace(0.1, 20, n, device="cuda").view(1, 1, n, 1).expand(1, 1, n, 128).half()
    bg.bgtq_fp4_append(ramp, torch.randn((1, 1, n, 128), device="cuda").half(), i32([0]), c.cache)
    c.q = torch.full((1, 4, t, 128), 0.5, device="cuda").half()
    c.check(c.run(False), False)
    c.q.neg_()
    c.check(c.run(False), False)


def test_tiny_values():
    """Values near the smallest that a block keeps come out at the same relative error."""
    c = Case(1, 4, 1, [500], 512, 0, seed=11)
    v = torch.randn((1, 1, 500, 128), device="cuda").mul_(1e-3).half()
    bg.bgtq_fp4_append(torch.randn((1, 1, 500, 128), device="cuda").half(), v, i32([0]), c.cache)
    c.check(c.run(False), False)


def test_three_dimensional_single_token():
    c = Case(2, 4, 1, [50, 9], 64, 0, seed=12, contiguous=True)
    want = c.run(True)
    out = torch.empty((2, 8, 128), dtype=torch.float16, device="cuda")
    ws = torch.zeros(bg.bgtq_fp4_attn_workspace(2, 4, 2, 1, 50), dtype=torch.uint8, device="cuda")
    bg.bgtq_fp4_attn(c.q.squeeze(2), c.cache, c.seq, 50, out, ws)
    assert torch.equal(out, want.squeeze(2))


def test_one_workspace_for_every_shape():
    """Calls of many shapes share a workspace in turn; each gives the bits of a call with a fresh one."""
    shapes = [(2, 8, 1, [9000, 20]), (1, 4, 1, [4000]), (2, 8, 4, [3000, 100]), (2, 2, 300, [2000, 301]), (2, 8, 1, [9000, 20]),
              (1, 1, 1, [1]), (2, 8, 30, [9000, 4000])]
    cases = [Case(H, G, t, lens, 9008, 0, seed=i) for i, (H, G, t, lens) in enumerate(shapes)]
    n = max(bg.bgtq_fp4_attn_workspace(c.H, c.G, len(c.lens), c.t, max(c.lens)) for c in cases)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    for c in cases + cases[::-1]:
        assert torch.equal(c.run(False, ws=ws), c.run(False))


def test_two_streams_with_two_workspaces():
    cs = [Case(2, 8, 1, [30000], 30016, 0, seed=1), Case(2, 8, 1, [30000], 30016, 0, seed=2)]
    want = [c.run(False) for c in cs]
    ws = [torch.zeros(bg.bgtq_fp4_attn_workspace(2, 8, 1, 1, 30000), dtype=torch.uint8, device="cuda") for _ in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    outs = [[], []]
    torch.cuda.synchronize()
    for _ in range(10):
        for i, c in enumerate(cs):
            with torch.cuda.stream(streams[i]):
                outs[i].append(c.run(False, ws=ws[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in outs[i])


def test_a_run_from_an_empty_cache():
    """A prompt in two chunks, then steps, all rotated on the way: every row against float64 over what the cache holds."""
    H, G, B = 2, 4, 2
    cap, page = 256, 32
    rope = bg.Rope(*bg.bgtq_rope_table(INV, 256))
    cache = new_cache(H, B, cap, page, spare=2, seed=13)
    ws = torch.zeros(bg.bgtq_fp4_attn_workspace(H, G, B, 100, cap), dtype=torch.uint8, device="cuda")
    n = np.array([0, 5])
    bg.bgtq_fp4_append(*(torch.randn((B, H, 5, 128), device="cuda").half() for _ in range(2)), i32([0, 0]), cache, rope=rope)
    for t, half in ((100, True), (37, False), (1, False), (1, True), (2, False), (1, False)):
        x = torch.randn((B, t, H * G + 2 * H, 128), device="cuda").half()
        q, k, v = (x[:, :, a:b].transpose(1, 2) for a, b in ((0, H * G), (H * G, H * G + H), (H * G + H, H * G + 2 * H)))
        start, n = n, n + t
        bg.bgtq_fp4_append(k, v, i32(start), cache, rope=rope)
        out = torch.empty((B, H * G, t, 128), dtype=torch.float16 if half else torch.float32, device="cuda")
        bg.bgtq_fp4_attn(q, cache, i32(n), cap, out, ws, rope=rope)
        c = Case.__new__(Case)
        c.H, c.G, c.t, c.lens, c.cache = H, G, t, n.tolist(), cache
        pos = i32(start[:, None] + np.arange(t))
        c.q = torch.empty((B, H * G, t, 128), dtype=torch.float16, device="cuda")
        bg.bgtq_rope_rows(rope, pos, q, c.q)
        c.check(out, half)


def test_a_captured_step_replayed():
    """Append and attend in a graph, lengths counted up on the device between replays; the graph beside an eager run."""
    H, G, B, cap = 2, 8, 2, 128
    rope = bg.Rope(*bg.bgtq_rope_table(INV, 256))
    a, b = new_cache(H, B, cap, 16, seed=14), new_cache(H, B, cap, 16, seed=14)
    k, v, q = (torch.randn((B, n, 1, 128), device="cuda").half() for n in (H, H, H * G))
    ws, ws2 = (torch.zeros(bg.bgtq_fp4_attn_workspace(H, G, B, 1, cap), dtype=torch.uint8, device="cuda") for _ in range(2))
    for c in (a, b):  # what the second sequence holds so far
        first = (torch.randn((B, H, 30, 128), device="cuda", generator=gen(i)).half() for i in (1, 2))
        bg.bgtq_fp4_append(*first, i32([0, 0]), c)
    start, n = i32([0, 30]), i32([1, 31])
    out, want = (torch.empty((B, H * G, 1, 128), device="cuda") for _ in range(2))

    def step(cache, o, w):
        bg.bgtq_fp4_append(k, v, start, cache, rope=rope)
        bg.bgtq_fp4_attn(q, cache, n, cap, o, w, rope=rope)

    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        step(a, out, ws)
    for _ in range(60):
        for x in (k, v, q):
            x.normal_()
        graph.replay()
        step(b, want, ws2)
        assert torch.equal(out, want) and torch.equal(a.groups, b.groups)
        start.add_(1)
        n.add_(1)


def test_python_refusals():
    c = Case(2, 4, 1, [20], 32, 0, seed=15)
    out = torch.empty((1, 8, 1, 128), device="cuda")
    ws = torch.zeros(bg.bgtq_fp4_attn_workspace(2, 4, 1, 1, 20), dtype=torch.uint8, device="cuda")
    rope = bg.Rope(*bg.bgtq_rope_table(INV, 64))
    good = dict(q=c.q, cache=c.cache, seq_lens=c.seq, max_len=20, out=out, workspace=ws)
    bg.bgtq_fp4_attn(**good)
    for bad in (dict(q=c.q[:, :7]), dict(q=c.q.float()), dict(out=out.double()), dict(out=out[:, :4]), dict(seq_lens=c.seq.long()),
                dict(seq_lens=c.seq.cpu()), dict(workspace=ws[:100]), dict(workspace=ws.cpu()), dict(pos=c.seq.view(1, 1)),
                dict(rope=rope, pos=c.seq.view(1, 1, 1).expand(2, 1, 1)), dict(q=torch.zeros((2, 8, 1, 128), dtype=torch.float16, device="cuda")),
                dict(q=torch.zeros((1, 18, 1, 128), dtype=torch.float16, device="cuda"))):
        with pytest.raises((ValueError, bg.BgtqError)):
            bg.bgtq_fp4_attn(**{**good, **bad})
    k = torch.zeros((1, 2, 3, 128), dtype=torch.float16, device="cuda")
    for bad in (dict(k=k.bfloat16()), dict(v=k[:, :, :2]), dict(pos_start=i32([0, 0])), dict(pos=i32([[0, 1, 2]])), dict(k=k[..., :64]),
                dict(k=k.cpu())):
        with pytest.raises(ValueError):
            bg.bgtq_fp4_append(**{**dict(k=k, v=k, pos_start=i32([0]), cache=c.cache), **bad})
    with pytest.raises(ValueError):
        bg.Fp4Cache(1, 1, 24)
    with pytest.raises(ValueError):
        bg.Fp4Cache(1, 1, 48, page_tokens=32)


def test_past_4_gigabytes_of_groups():
    """Groups at byte offsets past 2^32, and a sequence of more than 2^22 positions."""
    H, n = 8, (1 << 22) + 21
    cap = (n + 15) // 16 * 16
    cache = bg.Fp4Cache(H, 1, cap)
    assert cache.groups.numel() > 1 << 32
    cache.groups.view(-1, F.GROUP_BYTES)[:, 2048:] = 120  # scale 1; codes 0
    c = Case.__new__(Case)
    c.H, c.G, c.t, c.lens, c.cache, c.seq = H, 2, 1, [n], cache, i32([n])
    k, v = (torch.randn((1, H, 200, 128), device="cuda").half() * 30 for _ in range(2))
    bg.bgtq_fp4_append(k, v, i32([n - 200]), cache)
    c.q = torch.randn((1, 2 * H, 1, 128), device="cuda").half()
    out = c.run(False)
    got = out.double().cpu().numpy()
    at = group_rows(cache, 0, H - 1)[(n - 200) // 16:]
    raw = cache.groups.view(-1, F.GROUP_BYTES)[torch.from_numpy(at).cuda()].cpu().numpy()
    kc, ks, vc, vs = F.read(raw)
    off = (n - 200) % 16
    kk, vv = (F.fp4_value(x, s).reshape(-1, 128)[off:off + 200] for x, s in ((kc, ks), (vc, vs)))
    want_k, want_v = (F.fp4_value(*F.fp4_encode(x[0, H - 1].cpu().numpy())) for x in (k, v))
    assert np.array_equal(kk, want_k) and np.array_equal(vv, want_v)
    for a in (2 * H - 2, 2 * H - 1):
        x = c.q[0, a, 0].cpu().numpy().astype(np.float64)
        s = SCALE * kk @ x
        m = max(s.max(), 0.0)
        w = np.exp(s - m)
        total = w.sum() + (n - 200) * np.exp(-m)  # the other positions: keys and values 0
        want, mag = w @ vv / total, w @ np.abs(vv) / total
        d = SCALE * np.linalg.norm(x) * np.linalg.norm(kk, axis=1).max() * (2.0 ** -17 + 2.0 ** -22)
        # a warp's share is n / 16 / (304 / H * 8) groups: its sums' steps
        tol = (np.expm1(2 * d) + 2.0 ** -20 + (n / 16 / (304 // H * 8) + 400) * 2.0 ** -22) * mag
        tol = tol + 2.0 ** -33 * w.max() / total * np.abs(vv).sum(0)
        assert (np.abs(got[0, a, 0] - want) <= tol).all()
