"""The cases of the rotary operators and of the 4-bit cache: rotating queries
and keys by positions on one or several axes, appending un-rotated keys to the
packed Block-GTQ cache and to a cache of 4-bit values, and attention over the
latter; with their plain forms in elementary torch operations and their
definitions in 64 bits.

Operators (a case's "op"):
  rope         the queries and keys of a model's projection (a strided view)
               rotated into [B][heads][T][128]; one axis of positions or three
               (time, height, width); "inverse" is the rotation back, which is
               also its gradient
  rope_append  un-rotated keys rotated and quantize-appended, with their
               values, to the packed cache; the rotation's position is not the
               cache's slot (a cache that was cut keeps both apart)
  fp4_append   keys (rotated on the way) and values appended to the 4-bit cache
  fp4_attn     attention of T new rows (rotated on the way) over the 4-bit
               cache that holds them and everything before: T = 1 is a decode
               step, more a prompt's chunk

The bytes of a cache are its format's whole numbers: both sides have to write
the same ones.
"""

import functools
import math

import numpy as np
import torch

own = False

D = 128


def listed():
    return [
        # one token's heads of the one-KV-head layer: latency counts
        dict(name="rope_tiny", op="rope", B=1, T=1, H=1, G=4, axes=1, layout=0, n_pos=4096, dtype="f16", inverse=False),
        # a long prompt of the 128K layer
        dict(name="rope_long", op="rope", B=1, T=32768, H=2, G=8, axes=1, layout=0, n_pos=131072, dtype="f16", inverse=False),
        # two odd prompts with an image in them: positions on three axes, a projection in bf16
        dict(name="rope_axes", op="rope", B=2, T=4099, H=8, G=4, axes=3, layout=0, n_pos=32768, dtype="bf16", inverse=False),
        # one new token of every sequence of a ragged batch, paged
        dict(name="rope_append_step", op="rope_append", B=32, H=8, G=4, bk=2, bv=2, T=1, len_lo=1, len_hi=16384, cap=16384, page=256,
             axes=1, layout=0),
        # a prompt of 128K tokens into an empty cache
        dict(name="rope_append_long", op="rope_append", B=1, H=2, G=8, bk=3, bv=3, T=131072, len_lo=131072, len_hi=131072, cap=131072,
             page=0, axes=1, layout=0),
        # one new token of every sequence of a batch into the 4-bit cache
        dict(name="fp4_append_step", op="fp4_append", B=32, H=8, T=1, len_lo=1, len_hi=16384, cap=16384, page=256, axes=1, layout=0),
        # an odd long prompt, behind a few tokens
        dict(name="fp4_append_long", op="fp4_append", B=1, H=2, T=131043, len_lo=131064, len_hi=131064, cap=131072, page=0, axes=1, layout=0),
        # a decode step of the one-KV-head layer at 4K tokens
        dict(name="fp4_attn_tiny", op="fp4_attn", B=1, H=1, G=4, T=1, len_lo=4095, len_hi=4095, cap=4096, page=0, axes=1, layout=0,
             half=False),
        # a decode step of a ragged batch of 32, paged
        dict(name="fp4_attn_batch", op="fp4_attn", B=32, H=8, G=4, T=1, len_lo=1, len_hi=16384, cap=16384, page=256, axes=1, layout=0,
             half=True),
        # a decode step at 128K tokens
        dict(name="fp4_attn_long", op="fp4_attn", B=1, H=2, G=8, T=1, len_lo=131072, len_hi=131072, cap=131072, page=0, axes=1,
             layout=0, half=True),
        # a few drafted tokens checked at once at an odd length
        dict(name="fp4_attn_draft", op="fp4_attn", B=2, H=2, G=7, T=5, len_lo=50001, len_hi=50001, cap=65536, page=64, axes=1, layout=0,
             half=False),
        # a chunk of a long prompt
        dict(name="fp4_attn_chunk", op="fp4_attn", B=1, H=2, G=8, T=2048, len_lo=34815, len_hi=34815, cap=34816, page=0, axes=1, layout=0,
             half=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope_append", "fp4_append", "fp4_attn", "fp4_attn"])
    H, G = rng.choice([(1, 4), (2, 8), (8, 4), (4, 3), (3, 1), (2, 7)])
    case = dict(op=op, H=H, G=G, axes=rng.choice([1, 1, 3]), layout=rng.choice([0, 0, 1]))
    if op == "rope":
        B = _log_int(rng, 1, 32)
        T = _log_int(rng, 1, max(1, 32768 // (B * max(1, H * G // 16))))
        return dict(case, B=B, T=T, n_pos=max(T, _log_int(rng, 64, 131072)), dtype=rng.choice(["f16", "f16", "bf16", "f32"]),
                    inverse=rng.random() < 0.3)
    cap = max(16, _log_int(rng, 16, 131072) // 16 * 16)
    B = _log_int(rng, 1, max(1, min(32, (1 << 20) // (H * cap))))
    page = rng.choice([0, 0, 16, 64, 256])
    cap = -(-cap // page) * page if page else cap
    hi = rng.randint(max(1, cap // 2), cap)
    lo = rng.choice([1, hi])
    case.update(B=B, len_lo=lo, len_hi=hi, cap=cap, page=page)
    if op == "fp4_attn":
        T = min(lo, rng.choice([1, 1, 1, rng.randint(2, 16), _log_int(rng, 2, 2048)]))
        T = max(1, min(T, (1 << 30) // (B * H * G * hi)))
        return dict(case, T=T, half=T * G > 128 or rng.random() < 0.5)
    case.update(T=min(lo, rng.choice([1, _log_int(rng, 1, 131072)])))
    if op == "rope_append":
        bk, bv = rng.choice([(3, 3), (2, 2), (3, 2), (2, 4), (1, 3), (3, 1)])
        return dict(case, bk=bk, bv=bv)
    del case["G"]
    return case


# ----------------------------------------------------------------- the packed codec
# Block-GTQ as the cache holds it (widths by greedy gain, width classes cut
# into power-of-two rotation pieces, Lloyd-Max codes, four balanced lane
# slices per K record, token-pair V records).


def _sigma(head):
    sig = np.exp(1.2 * np.random.RandomState(1000 + head).standard_normal(64))
    sig[60:] *= 8.0
    return sig


def _signs(seed, head, tag):
    out = []
    for j in range(D):
        z = ((seed ^ (head << 16) ^ (tag << 8) ^ j) + 0x9E3779B97F4A7C15) & (2**64 - 1)
        z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & (2**64 - 1)
        z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & (2**64 - 1)
        out.append(-1.0 if (z ^ (z >> 31)) >> 63 else 1.0)
    return np.array(out)


def _lanes(wd, bk):
    """Bit position of codec pair m's field in the K record."""
    rank = {m: r for r, m in enumerate(sorted(range(64), key=lambda m: (-wd[m], m)))}
    left, lanes = list(range(64)), []
    for t in range(3):
        order = sorted(left, key=lambda m: ((rank[m] - t) % 4, rank[m]))
        can = [{(0, 0)}]  # can[i]: (items, bits) that the last i of `order` can make up
        for m in reversed(order):
            can.append(can[-1] | {(k + 1, s + wd[m]) for k, s in can[-1] if k < 16 and s + wd[m] <= 16 * bk})
        k, s, took = 16, 16 * bk, []
        for i, m in enumerate(order):
            if k and wd[m] <= s and (k - 1, s - wd[m]) in can[len(order) - i - 1]:
                took, k, s = took + [m], k - 1, s - wd[m]
        assert k == 0 and s == 0
        lanes.append(took)
        left = [m for m in left if m not in took]
    pos = np.zeros(64, np.int64)
    for t, lane in enumerate(lanes + [left]):
        a = sorted(lane, key=lambda m: (-wd[m], m))
        at = 32 * bk * t
        for m in a[0::2] + a[1::2]:
            pos[m] = at
            at += 2 * wd[m]
    return pos


@functools.lru_cache(maxsize=None)
def _codebooks():
    """Lloyd-Max levels of N(0, 1), widths 0..8: (levels rounded to fp16, midpoints), padded to 256."""
    cent, thr = np.zeros((9, 256)), np.full((9, 256), np.inf)
    for w in range(1, 9):
        n = 2**w
        half = np.sort(np.abs(np.random.RandomState(0).standard_normal(400000)))[np.arange(n // 2) * 400000 // (n // 2) + 200000 // n * 2]
        for _ in range(60 if w < 5 else 400):  # Newton's steps on the positive thresholds (the first is 0), damped while they are long
            t = np.concatenate([[0.0], 0.5 * (half[:-1] + half[1:]), [np.inf]])
            pdf = np.exp(-0.5 * np.minimum(t, 60) ** 2) / math.sqrt(2 * math.pi)
            mass = np.array([0.5 * (math.erfc(a / math.sqrt(2)) - math.erfc(b / math.sqrt(2))) for a, b in zip(t[:-1], t[1:])])
            mean = (pdf[:-1] - pdf[1:]) / mass
            fin = np.where(np.isfinite(t), t, 0.0)
            da, db = pdf[:-1] * (mean - fin[:-1]) / mass, pdf[1:] * (fin[1:] - mean) / mass
            k = len(half)
            jac = np.eye(k)
            for i in range(k):  # d mean_i / d half through the thresholds on both sides
                if i > 0:
                    jac[i, i - 1] -= 0.5 * da[i]
                    jac[i, i] -= 0.5 * da[i]
                if i < k - 1:
                    jac[i, i] -= 0.5 * db[i]
                    jac[i, i + 1] -= 0.5 * db[i]
            step = np.linalg.solve(jac, mean - half)
            scale = 1.0
            while np.any(np.diff(np.concatenate([[0.0], half + scale * step])) <= 0):
                scale *= 0.5
            half = half + scale * step
            if np.max(np.abs(step)) < 1e-13:
                break
        c = np.concatenate([-half[::-1], half]).astype(np.float16).astype(np.float64)
        cent[w, :n], thr[w, : n - 1] = c, 0.5 * (c[:-1] + c[1:])
    return cent, thr


@functools.lru_cache(maxsize=None)
def _tables(H, bk, bv, layout):
    """numpy tables of a layer's codec: [H][128] arrays in codec order."""
    seed, t = 0xB10C + 64 * bk + bv, {k: [] for k in ("bits", "energy", "perm", "width", "piece", "n", "white", "dewhite", "sk", "sv", "bit")}
    for h in range(H):
        s = 2.0 * _sigma(h) ** 2
        b = np.zeros(64, np.int64)
        for _ in range(64 * bk):
            b[np.argmax(np.where(b < 8, s * 0.25**b, -1.0))] += 1
        pieces = []
        for w in range(8, 0, -1):
            dims = [d for i in range(64) if b[i] == w for d in ((i, i + 64) if layout == 0 else (2 * i, 2 * i + 1))]
            at = 0
            for size in (128, 64, 32, 16, 8, 4, 2):
                if len(dims) & size:
                    pieces.append((size, w, dims[at : at + size]))
                    at += size
        pieces.sort(key=lambda p: (-p[0], -p[1]))
        perm = [d for p in pieces for d in p[2]]
        n = len(perm)
        perm += [d for d in range(D) if d not in perm]
        width = [p[1] for p in pieces for _ in p[2]] + [0] * (D - n)
        piece = [p[0] for p in pieces for _ in p[2]] + [1] * (D - n)
        pos = _lanes([width[2 * m] for m in range(64)], bk)
        e = s[np.array(perm) % 64 if layout == 0 else np.array(perm) // 2]
        for k, v in dict(bits=b, energy=s, perm=perm, width=width, piece=piece, n=n, white=np.sqrt(2.0 / e), dewhite=np.sqrt(e / 2.0),
                         sk=_signs(seed, h, 0), sv=_signs(seed, h, 1),
                         bit=[pos[j // 2] + (j % 2) * width[j] if width[j] else 0 for j in range(D)]).items():
            t[k].append(v)
    return seed, {k: np.array(v) for k, v in t.items()}


@functools.lru_cache(maxsize=None)
def _device_tables(H, bk, bv, layout):
    """The same on the GPU."""
    _, t = _tables(H, bk, bv, layout)
    _, thr = _codebooks()
    f32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.float32, device="cuda")  # noqa: E731
    i64 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int64, device="cuda")  # noqa: E731
    j = np.arange(D)
    return dict(thr=f32(thr), width=i64(t["width"]), bit=i64(t["bit"]), perm=i64(t["perm"]), piece=i64(t["piece"]), n=f32(t["n"]),
                white=f32(t["white"]), sk=f32(t["sk"]), sv=f32(t["sv"]), vbit=i64(np.stack([2 * bv * j, 2 * bv * j + bv])),
                coded=i64(t["width"]) > 0)


@functools.lru_cache(maxsize=None)
def _sigmas(H):
    return torch.tensor(np.stack([_sigma(h) for h in range(H)]), dtype=torch.float32, device="cuda")


@functools.lru_cache(maxsize=None)
def _plan(H, G, bk, bv, layout):
    """The framework's plan of that layer: made once for the layer, like a model's weights."""
    import rope_aware_quantized_gb300 as bg

    seed, t = _tables(H, bk, bv, layout)
    return bg.bgtq_plan_create(t["bits"], t["energy"], G, 128 * bk, bv, seed, rope_layout=layout)


# ----------------------------------------------------------------- packing
# Records as 32-bit words in int64; a code of `width` bits sits at bit `bit`.


def _pack(codes, bit, n_words):
    out = torch.zeros(*codes.shape[:-1], n_words + 1, dtype=torch.int64, device=codes.device)
    at, v = (bit >> 5).expand_as(codes), codes << (bit & 31)
    out.scatter_add_(-1, at, v & 0xFFFFFFFF)
    out.scatter_add_(-1, at + 1, v >> 32)
    out = out[..., :n_words]
    return (out - ((out >> 31) << 32)).to(torch.int32).view(torch.uint8)


def _slots(s, B, H, pos):
    """Record slot of positions pos [B, H, N] of every (sequence, head)."""
    b = torch.arange(B, device=pos.device).view(B, 1, 1)
    h = torch.arange(H, device=pos.device).view(1, H, 1)
    if s["table"] is None:
        return (b * H + h) * s["cap"] + pos
    P = s["page"]
    return (s["table"].to(torch.int64)[b, pos // P] * H + h) * P + pos % P


def _butterfly(x, h, piece):
    j = torch.arange(D, device=x.device)
    o = x[..., j ^ h]
    return torch.where(piece > h, torch.where((j & h) > 0, o - x, x + o), x)


def _encode(x, perm, white, sign, piece, n, coded, thr):
    """Codes and norms of rows x [..., N, 128] (fp32): one rounding an operation, in the order that the cache's format fixes."""
    z = torch.where(coded, x.gather(-1, perm.expand_as(x)) * white * sign, torch.zeros((), device=x.device))
    z = functools.reduce(lambda v, h: _butterfly(v, h, piece), (1, 2, 4, 8, 16, 32, 64), z)
    y = z * torch.tensor(1.0, device=x.device).div(piece.double().sqrt()).float()
    q = (y * y).view(*y.shape[:-1], 32, 4)
    q = (q[..., 0] + q[..., 1]) + (q[..., 2] + q[..., 3])
    lane = torch.arange(32, device=x.device)
    q = functools.reduce(lambda v, m: v + v[..., lane ^ m], (16, 8, 4, 2, 1), q)
    # quotients and the root through 64 bits: rounded once to 32 they are the correctly rounded ones
    rho = (q[..., :1].double() / n).float().double().sqrt().float()
    u = torch.where(rho > 0, (y.double() / torch.where(rho > 0, rho, torch.ones_like(rho))).float(), torch.zeros_like(y))
    u = u.movedim(-1, -2).contiguous()
    code = torch.searchsorted(thr.expand(*u.shape[:-1], thr.shape[-1]).contiguous(), u, right=True)
    return code.movedim(-2, -1), rho.squeeze(-1)


def _encode_kv(c, tab, k, v):
    w = lambda a: a.view(1, -1, 1, D)  # noqa: E731
    kc, kr = _encode(k.float(), w(tab["perm"]), w(tab["white"]), w(tab["sk"]), w(tab["piece"]), tab["n"].view(1, -1, 1, 1), w(tab["coded"]),
                     tab["thr"][tab["width"]].view(1, -1, D, 256))
    ident = torch.arange(D, device="cuda").view(1, 1, 1, D)
    one = torch.ones((), device="cuda")
    vc, vr = _encode(v.float(), ident, one, w(tab["sv"]), torch.full_like(ident, D), one * D, ident >= 0, tab["thr"][c["bv"]].view(1, 1, 1, 256))
    return torch.where(w(tab["coded"]), kc, torch.zeros_like(kc)), kr, vc, vr


# ----------------------------------------------------------------- the 4-bit cache
# Blocks of 16 values: a scale of 5 exponent and 3 mantissa bits (the bits
# 14..7 of an fp16 number) and 16 codes of e2m1.  The records of 16 positions
# of a head are one group of 2304 bytes: key codes (1024; a row's 64 bytes in
# the order [dim/4 mod 4][dim/16][dim mod 4]), value codes (1024; two
# neighbouring positions a byte, in the order [dim/64][dim mod 8][pos/2 mod 4]
# [dim/16 mod 4][pos/8][dim/8 mod 2]), key scales [pos][dim/16], value scales
# [pos/2 mod 4][dim/16][pos/8][pos mod 2].

GROUP = 2304


def _quantize(x):
    """Codes [..., 128] and scale bytes [..., 8] of rows x (fp32 values of fp16)."""
    blocks = x.unflatten(-1, (8, 16))
    y = blocks.abs().amax(-1) / 6
    e = (torch.frexp(y).exponent - 1).clamp_min(-14)
    step = torch.ldexp(torch.ones_like(y), e - 3)
    s = ((y / step).round() * step).clamp_max(10240)
    a, u = blocks.abs(), s.unsqueeze(-1)
    # the midpoints between neighbouring values; a tie goes to the even code (products exact in 32 bits)
    mag = (a > 0.25 * u).byte() + (a >= 0.75 * u) + (a > 1.25 * u) + (a >= 1.75 * u) + (a > 2.5 * u) + (a >= 3.5 * u) + (a > 5 * u)
    mag = torch.where(u > 0, mag, torch.zeros_like(mag))
    return (mag + 8 * torch.signbit(blocks).byte()).flatten(-2), (s.half().view(torch.int16) >> 7).byte()


def _nibbles(x):
    return x[..., 0] | (x[..., 1] << 4)


def _groups(kc, ks, vc, vs):
    """Codes [..., 16, 128] and scale bytes [..., 16, 8] of whole groups -> [..., 2304] bytes."""
    lead = kc.shape[:-2]
    n = len(lead)
    perm = lambda x, order: x.permute(*range(n), *[n + i for i in order])  # noqa: E731
    k = _nibbles(perm(kc.reshape(*lead, 16, 8, 4, 2, 2), (0, 2, 1, 3, 4)))
    v = _nibbles(perm(vc.reshape(*lead, 2, 4, 2, 2, 4, 2, 8), (3, 6, 1, 4, 0, 5, 2)))
    s = perm(vs.reshape(*lead, 2, 4, 2, 8), (1, 3, 0, 2))
    return torch.cat([x.reshape(*lead, -1) for x in (k, v, ks, s)], -1)


def _values(g):
    """Keys and values [..., 16, 128] (fp32) of whole groups [..., 2304]."""
    lead = g.shape[:-1]
    n = len(lead)
    perm = lambda x, order: x.permute(*range(n), *[n + i for i in order])  # noqa: E731
    two = lambda x: torch.stack([x & 15, x >> 4], -1)  # noqa: E731
    kc = perm(two(g[..., :1024]).reshape(*lead, 16, 4, 8, 2, 2), (0, 2, 1, 3, 4)).reshape(*lead, 16, 8, 16)
    vc = perm(two(g[..., 1024:2048]).reshape(*lead, 2, 8, 4, 4, 2, 2, 2), (4, 2, 6, 0, 3, 5, 1)).reshape(*lead, 16, 8, 16)
    ks = g[..., 2048:2176].reshape(*lead, 16, 8)
    vs = perm(g[..., 2176:].reshape(*lead, 4, 8, 2, 2), (2, 0, 3, 1)).reshape(*lead, 16, 8)
    level = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=g.device)
    scale = lambda s: (s.short() << 7).view(torch.float16).float().unsqueeze(-1)  # noqa: E731
    return (level[kc.int()] * scale(ks)).flatten(-2), (level[vc.int()] * scale(vs)).flatten(-2)


def _group_at(s, B, H, i):
    """Index of group i [B, 1, N] of every (sequence, head)."""
    b = torch.arange(B, device="cuda").view(B, 1, 1)
    h = torch.arange(H, device="cuda").view(1, H, 1)
    if s["table"] is None:
        return (b * H + h) * (s["cap"] // 16) + i
    P = s["page"] // 16
    return (s["table"].to(torch.int64)[b, i // P] * H + h) * P + i % P


# ----------------------------------------------------------------- inputs


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


@functools.lru_cache(maxsize=2)
def _rope_tables(n_pos):
    """cos and sin [n_pos][64] of base 10^6, angles in 64 bits."""
    a = torch.arange(n_pos, device="cuda", dtype=torch.float64).unsqueeze(1) * 1e6 ** (-torch.arange(64, device="cuda", dtype=torch.float64) / 64)
    return a.cos().float(), a.sin().float()


def _axis(c):
    """Axis of each of the 64 frequencies: time in the first 16, height and width in 24 each."""
    return [0] * 16 + [1] * 24 + [2] * 24 if c["axes"] == 3 else [0] * 64


def _image(T):
    """Tokens of text before the image, and its width."""
    text = T // 4
    return text, max(1, math.isqrt(T - text))


def _positions(c, first):
    """[axes][B][T] positions from first [B] on; on three axes some text, then an image in rows."""
    t = torch.arange(c["T"], device="cuda")
    if c["axes"] == 3:
        text, side = _image(c["T"])
        i = (t - text).clamp_min(0)
        t = torch.stack([t.clamp_max(text), t.clamp_max(text) + i // side, t.clamp_max(text) + i % side])
    return (first.view(1, -1, 1) + t.view(c["axes"], 1, -1)).to(torch.int32).contiguous()


def _lens(c, g):
    n = torch.randint(c["len_lo"], c["len_hi"] + 1, (c["B"],), device="cuda", generator=g, dtype=torch.int32)
    n[0] = c["len_hi"]
    return n


def _table(c, g):
    if not c["page"]:
        return None
    return torch.randperm(c["B"] * c["cap"] // c["page"], device="cuda", generator=g).to(torch.int32).view(c["B"], -1)


def _projection(c, g, nq, H, dtype=torch.float16):
    """What a layer's projection gives: [B][T][nq + 2 H][128], keys and queries with each rotary block's spread; -> q, k, v as views [B][heads][T][128]."""
    x = torch.randn((c["B"], c["T"], nq + 2 * H, D), device="cuda", generator=g, dtype=torch.float32)
    s = _sigmas(H)
    spread = lambda w: torch.cat([w, w], -1) if c["layout"] == 0 else w.repeat_interleave(2, -1)  # noqa: E731
    if nq:  # logits that spread by about 2, as trained heads' do
        logit = (2 * s.double().pow(4).sum(-1, keepdim=True)).sqrt().float() / math.sqrt(D)
        x[:, :, :nq] *= spread(s * (2.0 / logit)).repeat_interleave(nq // H, 0)
    x[:, :, nq : nq + H] *= spread(s)
    x = x.to(dtype).transpose(1, 2)
    return x[:, :nq], x[:, nq : nq + H], x[:, nq + H :]


def prepare(case, seed):
    c, g = dict(case), _generator(seed)
    B, T, H = c["B"], c["T"], c["H"]
    st = dict(c=c)
    st["cos"], st["sin"] = _rope_tables(c["n_pos"] if c["op"] == "rope" else c["cap"])
    if own:  # the handle that a user's program keeps for its tables
        import rope_aware_quantized_gb300 as bg

        st["rope"] = bg.Rope(st["cos"], st["sin"], layout=c["layout"], axis=_axis(c))
    if c["op"] == "rope":
        dtype = dict(f16=torch.float16, bf16=torch.bfloat16, f32=torch.float32)[c["dtype"]]
        st["q"], st["k"], _ = _projection(c, g, H * c["G"], H, dtype)
        st["pos"] = _positions(c, torch.randint(0, c["n_pos"] - T + 1, (B,), device="cuda", generator=g))
        st["q_out"] = torch.empty(st["q"].shape, dtype=torch.float16, device="cuda")
        st["k_out"] = torch.empty(st["k"].shape, dtype=torch.float16, device="cuda")
        return st
    st["lens"] = _lens(c, g)
    st["first"] = (st["lens"] - T).to(torch.int32)
    st["pos"] = _positions(c, st["first"])
    st["table"] = _table(c, g)
    st.update(cap=c["cap"], page=c["page"])
    if c["op"] == "rope_append":
        _, st["k"], st["v"] = _projection(c, g, 0, H)
        rows = B * H * c["cap"]
        byte = lambda n: torch.randint(0, 256, (n,), device="cuda", generator=g, dtype=torch.uint8)  # noqa: E731
        st.update(k_codes=byte(rows * 16 * c["bk"]), v_codes=byte(rows * 16 * c["bv"]), k_norm=torch.ones(rows, device="cuda"),
                  v_norm=torch.ones(rows, device="cuda"))
        if own:
            st["plan"] = _plan(H, c["G"], c["bk"], c["bv"], c["layout"])
            st["cache"] = bg.Cache(st["plan"], B, c["cap"], page_tokens=c["page"])
            list(map(lambda n: getattr(st["cache"], n).copy_(st[n]), ("k_codes", "v_codes", "k_norm", "v_norm")))
            if c["page"]:
                st["cache"].page_table.copy_(st["table"])
        return st
    # what the sequences hold so far: keys with each block's spread, values near Gaussian
    shape = (B, H, c["cap"] // 16, 16, D)
    s = _sigmas(H)
    k = torch.randn(shape, device="cuda", generator=g).mul_(torch.cat([s, s], -1).view(1, H, 1, 1, D)).half().float()
    v = torch.randn(shape, device="cuda", generator=g).half().float()
    groups = _groups(*_quantize(k), *_quantize(v))
    del k, v
    st["groups"] = torch.empty_like(groups)
    at = _group_at(st, B, H, torch.arange(c["cap"] // 16, device="cuda").view(1, 1, -1))
    st["groups"].view(-1, GROUP)[at] = groups
    del groups
    if own:
        st["cache"] = bg.Fp4Cache(H, B, c["cap"], page_tokens=c["page"])
        st["cache"].groups.copy_(st["groups"].view(-1))
        if c["page"]:
            st["cache"].page_table.copy_(st["table"])
    if c["op"] == "fp4_append":
        _, st["k"], st["v"] = _projection(c, g, 0, H)
        return st
    st["q"], _, _ = _projection(c, g, H * c["G"], H)
    st["out"] = torch.empty(st["q"].shape, dtype=torch.float16 if c["half"] else torch.float32, device="cuda")
    if own:
        n = bg.bgtq_fp4_attn_workspace(H, c["G"], B, T, c["len_hi"])
        st["ws"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
    return st


# ----------------------------------------------------------------- the calls


def run(st):
    c = st["c"]
    if own:
        return _run_own(c, st)
    return {"rope": _rope, "rope_append": _rope_append, "fp4_append": _fp4_append, "fp4_attn": _fp4_attn}[c["op"]](c, st)


def _run_own(c, st):
    import rope_aware_quantized_gb300 as bg

    if c["op"] == "rope":
        bg.bgtq_rope_rows(st["rope"], st["pos"], st["q"], st["q_out"], st["k"], st["k_out"], inverse=c["inverse"])
        return dict(q=st["q_out"], k=st["k_out"])
    if c["op"] == "rope_append":
        bg.bgtq_rope_append(st["plan"], st["rope"], st["pos"], st["k"], st["v"], st["first"], st["cache"])
        return {n: getattr(st["cache"], n) for n in ("k_codes", "v_codes", "k_norm", "v_norm")}
    if c["op"] == "fp4_append":
        bg.bgtq_fp4_append(st["k"], st["v"], st["first"], st["cache"], rope=st["rope"], pos=st["pos"])
        return dict(groups=st["cache"].groups)
    bg.bgtq_fp4_attn(st["q"], st["cache"], st["lens"], c["len_hi"], st["out"], st["ws"], rope=st["rope"], pos=st["pos"])
    return dict(out=st["out"])


# ----------------------------------------------------------------- plain forms


def _rotate(c, st, x, inverse=False):
    """Rows x [B][heads][T][128] rotated, in 32 bits: each product and the sum rounded."""
    i = torch.arange(64, device="cuda")
    p = st["pos"].to(torch.int64)[torch.tensor(_axis(c), device="cuda")].permute(1, 2, 0)  # [B][T][64]
    cos, sin = st["cos"][p, i].unsqueeze(1), st["sin"][p, i].unsqueeze(1)
    sin = -sin if inverse else sin
    x = x.float()
    lo, hi = (x[..., :64], x[..., 64:]) if c["layout"] == 0 else (x[..., 0::2], x[..., 1::2])
    lo, hi = lo * cos - hi * sin, hi * cos + lo * sin
    return torch.cat([lo, hi], -1) if c["layout"] == 0 else torch.stack([lo, hi], -1).flatten(-2)


def _rope(c, st):
    return dict(q=_rotate(c, st, st["q"], c["inverse"]).half(), k=_rotate(c, st, st["k"], c["inverse"]).half())


def _rope_append(c, st):
    B, H, T = c["B"], c["H"], c["T"]
    tab = _device_tables(H, c["bk"], c["bv"], c["layout"])
    kc, kr, vc, vr = _encode_kv(c, tab, _rotate(c, st, st["k"]).half(), st["v"])
    pos = (st["first"].to(torch.int64).view(-1, 1, 1) + torch.arange(T, device="cuda")).expand(B, H, T)
    slot = _slots(st, B, H, pos)
    st["k_codes"].view(-1, 16 * c["bk"])[slot] = _pack(kc, tab["bit"].view(1, -1, 1, D), 4 * c["bk"])
    st["k_norm"][slot] = kr
    st["v_norm"][slot] = vr
    # a V record holds two positions: whole pairs from the first one's, the half that is not appended stays
    e = (st["first"].to(torch.int64) & 1).view(-1, 1, 1)
    at = 2 * torch.arange(T // 2 + 1, device="cuda").view(1, 1, -1, 1) + torch.arange(2, device="cuda") - e.unsqueeze(-1)
    new = (at >= 0) & (at < T)
    codes = vc.gather(2, at.clamp(0, T - 1).view(B, 1, -1, 1).expand(B, H, -1, D)).view(B, H, -1, 2, D)
    zero = torch.zeros_like(codes)
    put = lambda x: _pack(torch.where(new.unsqueeze(-1), x, zero).flatten(-2), tab["vbit"].reshape(-1), 8 * c["bv"])  # noqa: E731
    mask, rec = put(zero + (2 ** c["bv"] - 1)), put(codes)
    pair = pos[..., :1] - e + 2 * torch.arange(T // 2 + 1, device="cuda")
    some = new.any(-1).expand(B, H, -1)
    pair = (_slots(st, B, H, pair.clamp_max(c["cap"] - 1)) >> 1)[some]
    pairs = st["v_codes"].view(-1, 32 * c["bv"])
    pairs[pair] = (pairs[pair] & ~mask.expand(B, H, -1, -1)[some]) | rec[some]
    return {n: st[n] for n in ("k_codes", "v_codes", "k_norm", "v_norm")}


def _fp4_append(c, st):
    B, H, T = c["B"], c["H"], c["T"]
    kc, ks = _quantize(_rotate(c, st, st["k"]).half().float())
    vc, vs = _quantize(st["v"].float())
    first = st["first"].to(torch.int64).view(-1, 1)
    n = (T + 14) // 16 + 1  # groups that T rows can touch
    at = 16 * (first // 16) + torch.arange(16 * n, device="cuda") - first  # row of every position of those groups [B, 16 n]
    new = ((at >= 0) & (at < T)).view(B, 1, 16 * n, 1)
    row = at.clamp(0, T - 1).view(B, 1, -1, 1)
    take = lambda x: torch.where(new, x.gather(2, row.expand(B, H, -1, x.shape[-1])), torch.zeros_like(x[:, :, :1, :1])).unflatten(2, (n, 16))  # noqa: E731
    ones = lambda v, w: (new * v).byte().expand(B, H, -1, w).unflatten(2, (n, 16))  # noqa: E731
    rec, mask = _groups(take(kc), take(ks), take(vc), take(vs)), _groups(ones(15, D), ones(255, 8), ones(15, D), ones(255, 8))
    some = new.view(B, 1, n, 16).any(-1).expand(B, H, -1)
    i = (first // 16).view(B, 1, 1) + torch.arange(n, device="cuda")
    slot = _group_at(st, B, H, i.clamp_max(c["cap"] // 16 - 1))[some]
    groups = st["groups"].view(-1, GROUP)
    groups[slot] = (groups[slot] & ~mask[some]) | rec[some]
    return dict(groups=st["groups"].view(-1))


def _fp4_attn(c, st):
    B, H, G, T, N = c["B"], c["H"], c["G"], c["T"], -(-c["len_hi"] // 16)
    at = _group_at(st, B, H, torch.arange(N, device="cuda").view(1, 1, -1))
    k, v = _values(st["groups"].view(-1, GROUP)[at])
    k, v = k.flatten(2, 3), v.flatten(2, 3)  # [B, H, 16 N, 128]
    q = _rotate(c, st, st["q"]).half().float().view(B, H, G * T, D)
    row = st["first"].view(-1, 1, 1, 1) + torch.arange(T, device="cuda").repeat(G).view(1, 1, -1, 1)
    seen = torch.arange(16 * N, device="cuda") <= row
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(1 / math.sqrt(D)).masked_fill_(~seen, -math.inf)
    p = s.sub_(s.amax(-1, keepdim=True).clamp_min(-1e30)).exp_()
    out = torch.matmul(p, v) / p.sum(-1, keepdim=True).clamp_min(1e-30)
    return dict(out=out.view(st["out"].shape).to(st["out"].dtype))


# ----------------------------------------------------------------- the floors


def _mean(c):
    """Positions of all sequences together (the first is the longest, the others uniform)."""
    return c["len_hi"] + (c["B"] - 1) * (c["len_lo"] + c["len_hi"]) / 2


def _table_bytes(c, n_pos):
    """cos and sin rows that the positions meet, and the positions."""
    text, side = _image(c["T"])
    rows = c["T"] if c["axes"] == 1 else text + side
    return 512 * min(n_pos, c["B"] * rows) + 4 * c["axes"] * c["B"] * c["T"]


def work(case):
    c = case
    B, T, H = c["B"], c["T"], c["H"]
    rows = B * T * H
    if c["op"] == "rope":
        n = B * T * H * (c["G"] + 1)
        return dict(bytes=n * D * ((4 if c["dtype"] == "f32" else 2) + 2) + _table_bytes(c, c["n_pos"]), flops=3 * D * n)
    table = _table_bytes(c, c["cap"])
    if c["op"] == "rope_append":
        return dict(bytes=rows * (512 + 16 * c["bk"] + 16 * c["bv"] + 8) + table, flops=rows * D * (3 + 2 * 14))
    if c["op"] == "fp4_append":
        return dict(bytes=rows * (512 + 144) + table, flops=rows * D * (3 + 2 * 4))
    pairs = T * (_mean(c) - c["B"] * (T - 1) / 2)
    q = B * T * H * c["G"] * D
    return dict(bytes=H * _mean(c) * 144 + q * (2 + (2 if c["half"] else 4)) + table, flops=4 * D * H * c["G"] * pairs)


# ----------------------------------------------------------------- 64 bits


def _rotate64(c, st, x):
    axis = _axis(c)
    out = torch.empty(x.shape, dtype=torch.float64, device="cuda")
    sign = -1.0 if c.get("inverse") else 1.0
    for i in range(64):
        a, b = (i, i + 64) if c["layout"] == 0 else (2 * i, 2 * i + 1)
        p = st["pos"][axis[i]].long()
        z = torch.complex(x[..., a].double(), x[..., b].double())
        z = z * torch.complex(st["cos"][:, i].double(), sign * st["sin"][:, i].double())[p].unsqueeze(1)
        out[..., a], out[..., b] = z.real, z.imag
    return out


def _norm64(x, white):
    """Root mean square of whitened coordinates (the rotation keeps it)."""
    n = int((white > 0).sum())
    return ((x.double() * white).pow(2).sum(-1) / n).sqrt()


def exact(case, seed):
    c, st = case, prepare(case, seed)
    B, T, H = c["B"], c["T"], c["H"]
    if c["op"] == "rope":
        return dict(q=_rotate64(c, st, st["q"]), k=_rotate64(c, st, st["k"]))
    if c["op"] == "fp4_append":
        return None  # writes whole numbers: nothing of it is kept in floating point
    if c["op"] == "rope_append":
        k = _rotate64(c, st, st["k"]).half()  # the cached key is an fp16 number
        _, t = _tables(H, c["bk"], c["bv"], c["layout"])
        k_norm, v_norm = st["k_norm"].double(), st["v_norm"].double()
        for b in range(B):
            pos = int(st["first"][b]) + torch.arange(T, device="cuda")
            for h in range(H):
                w = torch.zeros(D, dtype=torch.float64, device="cuda")
                m = int(t["n"][h])
                w[torch.tensor(t["perm"][h][:m], device="cuda")] = torch.tensor(t["white"][h][:m], device="cuda")
                if st["table"] is None:
                    slot = (b * H + h) * c["cap"] + pos
                else:
                    slot = (st["table"][b, pos // c["page"]].long() * H + h) * c["page"] + pos % c["page"]
                k_norm[slot] = _norm64(k[b, h], w)
                v_norm[slot] = _norm64(st["v"][b, h], torch.ones_like(w))
        return dict(k_codes=None, v_codes=None, k_norm=k_norm, v_norm=v_norm)
    G = c["G"]
    q = _rotate64(c, st, st["q"]).half().double()  # the rotated query is an fp16 number
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    grid = torch.cat([grid, -grid])
    d, raw = torch.arange(D, device="cuda"), st["groups"].view(-1)
    for b in range(B):
        n = int(st["lens"][b])
        j = torch.arange(n, device="cuda").unsqueeze(1)
        t = j % 16
        for h in range(H):
            if st["table"] is None:
                at = (b * H + h) * (c["cap"] // 16) + j // 16
            else:
                at = (st["table"][b, j // c["page"]].long() * H + h) * (c["page"] // 16) + j % c["page"] // 16
            at = at * GROUP
            # each value's own byte and scale, as the layout above says
            kb = raw[at + 64 * t + 16 * (d // 4 % 4) + 2 * (d // 16) + d // 2 % 2] >> (4 * (d % 2)).byte()
            vb = raw[at + 1024 + 512 * (d // 64) + 64 * (d % 8) + 16 * (t // 2 % 4) + 4 * (d // 16 % 4) + 2 * (t // 8) + d // 8 % 2]
            vb = vb >> (4 * (t % 2)).byte()
            ks = raw[at + 2048 + 8 * t + d // 16]
            vs = raw[at + 2176 + 32 * (t // 2 % 4) + 4 * (d // 16) + 2 * (t // 8) + t % 2]
            number = lambda s: torch.where(s < 8, s * 2.0**-17, (8 + s % 8) * 2.0 ** (s // 8 - 18.0))  # noqa: E731
            k = grid[(kb & 15).long()] * number(ks.double())
            v = grid[(vb & 15).long()] * number(vs.double())
            for a in range(h * G, (h + 1) * G):
                s = q[b, a] @ k.T / math.sqrt(D)
                late = torch.arange(n, device="cuda") > (n - T + torch.arange(T, device="cuda")).unsqueeze(1)
                out[b, a] = s.masked_fill(late, -math.inf).softmax(-1) @ v
    return dict(out=out)
