"""The cases of the bounded-cache operators: attention with a sliding window and
sinks, accumulated attention weights, and eviction by them, on the packed
Block-GTQ cache; with their plain forms in elementary torch operations and
their definitions in 64 bits.

Operators (a case's "op"):
  window_decode   one token's attention over the packed cache, restricted to
                  the first `sinks` and the last `window` positions; with
                  "step" the token is quantize-appended first
  window_prefill  causal attention of a prompt under the same restriction, its
                  log-sum-exp and its packed records
  score_decode    one token's attention over the whole packed cache, its
                  weights added to every cached position's score
  score_prefill   the weights that a prompt's rows from row0 on give to every
                  position, from the log-sum-exp of the prefill
  evict           the best `keep` positions of every (sequence, KV head) by
                  score (the first `sinks` and the last `recent` always), moved
                  into another packed cache
"""

import functools
import math

import numpy as np
import torch

own = False

D = 128


def listed():
    return [
        # the smallest call: one sequence of the one-KV-head test layer, short window; latency counts
        dict(name="window_decode_tiny", op="window_decode", B=1, H=1, G=4, bk=3, bv=3, len_lo=1537, len_hi=1537, cap=4096,
             page=0, sinks=4, window=251, step=False, half=False),
        # a serving batch: 32 ragged sequences on a paged cache, the step of every layer
        dict(name="window_decode_batch", op="window_decode", B=32, H=8, G=4, bk=2, bv=2, len_lo=1, len_hi=16384, cap=16384,
             page=256, sinks=16, window=4096, step=True, half=True),
        # a long context of 128K tokens read through a wide, odd window
        dict(name="window_decode_long", op="window_decode", B=1, H=2, G=8, bk=3, bv=3, len_lo=131071, len_hi=131071,
             cap=131072, page=0, sinks=100, window=65535, step=False, half=False),
        # two short prompts of odd length under a narrow window
        dict(name="window_prefill_odd", op="window_prefill", B=2, H=2, G=8, bk=3, bv=3, T=1531, sinks=5, window=255),
        # a long prompt under the usual window
        dict(name="window_prefill_long", op="window_prefill", B=1, H=2, G=8, bk=3, bv=3, T=32768, sinks=4, window=4096),
        # scores of one step of the one-KV-head layer
        dict(name="score_decode_tiny", op="score_decode", B=1, H=1, G=4, bk=3, bv=3, len_lo=4095, len_hi=4095, cap=4096,
             page=0, step=True, half=False),
        # scores of one step at 128K tokens
        dict(name="score_decode_long", op="score_decode", B=1, H=2, G=8, bk=3, bv=3, len_lo=131072, len_hi=131072,
             cap=131072, page=0, step=True, half=True),
        # the last 64 rows of a long prompt rank its positions before the cache is cut to a budget
        dict(name="score_prefill_rows", op="score_prefill", B=1, H=8, G=4, T=32768, row0=32704, sinks=0, window=32768),
        # every row of a prompt counts
        dict(name="score_prefill_all", op="score_prefill", B=1, H=2, G=8, T=8191, row0=0, sinks=0, window=8191),
        # a short cache cut to a quarter
        dict(name="evict_tiny", op="evict", B=1, H=1, bk=3, bv=3, len_lo=4001, len_hi=4001, cap=4096, page=0, keep=1021,
             sinks=4, recent=64),
        # a 128K cache cut to 32K
        dict(name="evict_long", op="evict", B=1, H=2, bk=3, bv=3, len_lo=131072, len_hi=131072, cap=131072, page=0,
             keep=32768, sinks=4, recent=1024),
        # a ragged paged batch cut to 4K each; the short sequences are kept whole
        dict(name="evict_batch", op="evict", B=32, H=8, bk=2, bv=2, len_lo=1, len_hi=16384, cap=16384, page=256, keep=4095,
             sinks=16, recent=256),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["window_decode", "window_prefill", "score_decode", "score_prefill", "evict"])
    H, G = rng.choice([(1, 4), (2, 8), (8, 4), (4, 3), (3, 1), (2, 7)])
    bk, bv = rng.choice([(3, 3), (2, 2), (3, 2), (2, 4), (1, 3), (3, 1)])
    if op in ("window_decode", "score_decode", "evict"):
        cap = max(16, _log_int(rng, 16, 131072) // 2 * 2)
        B = _log_int(rng, 1, max(1, min(32, (1 << 20) // (H * cap))))
        page = rng.choice([0, 0, 16, 64, 256])
        cap = -(-cap // page) * page if page else cap
        hi = rng.randint(max(1, cap // 2), cap)
        case = dict(op=op, B=B, H=H, G=G, bk=bk, bv=bv, len_lo=rng.choice([1, hi]), len_hi=hi, cap=cap, page=page)
        if op == "evict":
            del case["G"]
            keep = _log_int(rng, 1, cap)
            sinks = rng.randint(0, min(keep, 64))
            return dict(case, keep=keep, sinks=sinks, recent=rng.randint(0, min(keep - sinks, 1024)))
        case.update(step=rng.random() < 0.5, half=rng.random() < 0.5)
        if op == "window_decode":
            case.update(sinks=rng.choice([0, 1, 4, 17, 128]), window=_log_int(rng, 1, cap))
        return case
    B = rng.choice([1, 1, 2, 3])
    if op == "window_prefill":
        T = _log_int(rng, 1, 16384 // B)
        return dict(op=op, B=B, H=H, G=G, bk=bk, bv=bv, T=T, sinks=rng.choice([0, 1, 4, 17, 130]),
                    window=_log_int(rng, 1, max(1, min(T, 4096))))
    T = _log_int(rng, 1, 32768 // B)
    rows = _log_int(rng, 1, max(1, min(T, (1 << 26) // (B * T))))
    return dict(op=op, B=B, H=H, G=G, T=T, row0=T - rows, sinks=rng.choice([0, 4, 17]),
                window=rng.choice([T, T, _log_int(rng, 1, T)]))


# ----------------------------------------------------------------- the codec
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
def _tables(H, bk, bv):
    """numpy tables of a layer's codec: [H][128] arrays in codec order."""
    seed, t = 0xB10C + 64 * bk + bv, {k: [] for k in ("bits", "energy", "perm", "width", "piece", "n", "white", "dewhite", "sk", "sv", "bit")}
    for h in range(H):
        s = 2.0 * _sigma(h) ** 2
        b = np.zeros(64, np.int64)
        for _ in range(64 * bk):
            b[np.argmax(np.where(b < 8, s * 0.25**b, -1.0))] += 1
        pieces = []
        for w in range(8, 0, -1):
            dims = [d for i in range(64) if b[i] == w for d in (i, i + 64)]
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
        e = s[np.array(perm) % 64]
        for k, v in dict(bits=b, energy=s, perm=perm, width=width, piece=piece, n=n, white=np.sqrt(2.0 / e), dewhite=np.sqrt(e / 2.0),
                         sk=_signs(seed, h, 0), sv=_signs(seed, h, 1),
                         bit=[pos[j // 2] + (j % 2) * width[j] if width[j] else 0 for j in range(D)]).items():
            t[k].append(v)
    return seed, {k: np.array(v) for k, v in t.items()}


@functools.lru_cache(maxsize=None)
def _hadamard(n):
    h = np.ones((1, 1))
    while len(h) < n:
        h = np.block([[h, h], [h, -h]])
    return h


@functools.lru_cache(maxsize=None)
def _device_tables(H, bk, bv):
    """The same on the GPU, with the matrices that take a codec row to its dims: khat = y @ rk[h], vhat = y @ rv[h]."""
    seed, t = _tables(H, bk, bv)
    rk, rv = np.zeros((H, D, D)), np.zeros((H, D, D))
    for h in range(H):
        j = 0
        while j < t["n"][h]:
            p = int(t["piece"][h][j])
            at = np.arange(j, j + p)
            f = (t["sk"][h][at] * t["dewhite"][h][at]) / math.sqrt(p)
            rk[h][np.ix_(at, t["perm"][h][at])] = _hadamard(p) * f[None, :]
            j += p
        rv[h] = _hadamard(D) * t["sv"][h][None, :] / math.sqrt(D)
    cent, thr = _codebooks()
    f32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.float32, device="cuda")  # noqa: E731
    i64 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int64, device="cuda")  # noqa: E731
    j = np.arange(D)
    return dict(rk=f32(rk), rv=f32(rv), cent=f32(cent), thr=f32(thr), width=i64(t["width"]), bit=i64(t["bit"]), perm=i64(t["perm"]),
                piece=i64(t["piece"]), n=f32(t["n"]), white=f32(t["white"]), sk=f32(t["sk"]), sv=f32(t["sv"]),
                vbit=i64(np.stack([2 * bv * j, 2 * bv * j + bv])), coded=i64(t["width"]) > 0,
                sigma=f32(np.sqrt(t["energy"] / 2.0)))


@functools.lru_cache(maxsize=None)
def _plan(H, G, bk, bv):
    """The framework's plan of that layer: made once for the layer, like a model's weights."""
    import rope_aware_quantized_gb300 as bg

    seed, t = _tables(H, bk, bv)
    return bg.bgtq_plan_create(t["bits"], t["energy"], G, 128 * bk, bv, seed)


# ----------------------------------------------------------------- packing
# Records as 32-bit words in int64; a code of `width` bits sits at bit `bit`.


def _words(rec):
    w = rec.contiguous().view(torch.int32).to(torch.int64) & 0xFFFFFFFF
    return torch.nn.functional.pad(w, (0, 1))


def _fields(words, bit, width):
    at = (bit >> 5).expand(*words.shape[:-1], bit.shape[-1])
    return ((words.gather(-1, at) | (words.gather(-1, at + 1) << 32)) >> (bit & 31)) & ((1 << width) - 1)


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


def _dequant(c, tab, s, pos):
    """The cached keys and values at positions pos [B, H, N] -> [B, H, N, 128] each."""
    slot = _slots(s, c["B"], c["H"], pos)
    kw = _words(s["k_codes"].view(-1, 16 * c["bk"])[slot])
    kcode = _fields(kw, tab["bit"].view(1, -1, 1, D), tab["width"].view(1, -1, 1, D))
    ky = tab["cent"][tab["width"].view(1, -1, 1, D), kcode] * s["k_norm"].view(-1)[slot].unsqueeze(-1)
    vw = _words(s["v_codes"].view(-1, 32 * c["bv"])[slot >> 1])
    vcode = _fields(vw, tab["vbit"][slot & 1], torch.tensor(c["bv"], device="cuda"))
    vy = tab["cent"][c["bv"]][vcode] * s["v_norm"].view(-1)[slot].unsqueeze(-1)
    return ky @ tab["rk"], vy @ tab["rv"]


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


def _append(c, tab, s, k_new, v_new, pos_new):
    """The new token [B, H, 128] of every sequence into the cache."""
    kc, kr, vc, vr = _encode_kv(c, tab, k_new.unsqueeze(2), v_new.unsqueeze(2))
    slot = _slots(s, c["B"], c["H"], pos_new.to(torch.int64).view(-1, 1, 1).expand(-1, c["H"], 1))
    s["k_codes"].view(-1, 16 * c["bk"])[slot] = _pack(kc, tab["bit"].view(1, -1, 1, D), 4 * c["bk"])
    s["k_norm"].view(-1)[slot] = kr
    s["v_norm"].view(-1)[slot] = vr
    pairs = s["v_codes"].view(-1, 32 * c["bv"])
    bits = tab["vbit"][slot & 1]
    full = torch.full_like(vc, 2 ** c["bv"] - 1)
    pairs[slot >> 1] = (pairs[slot >> 1] & ~_pack(full, bits, 8 * c["bv"])) | _pack(vc, bits, 8 * c["bv"])


# ----------------------------------------------------------------- inputs


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _lens(c, g):
    n = torch.randint(c["len_lo"], c["len_hi"] + 1, (c["B"],), device="cuda", generator=g, dtype=torch.int32)
    n[0] = c["len_hi"]
    return n


def _cache(c, g, cap, page):
    """Descriptor of an empty packed cache: contiguous, or pools of pages in a shuffled order."""
    rows, table = c["B"] * c["H"] * cap, None
    if page:
        table = torch.randperm(c["B"] * cap // page, device="cuda", generator=g).to(torch.int32).view(c["B"], -1)
    z = lambda n, t: torch.zeros(n, dtype=t, device="cuda")  # noqa: E731
    return dict(k_codes=z(rows * 16 * c["bk"], torch.uint8), v_codes=z(rows * 16 * c["bv"], torch.uint8), k_norm=z(rows, torch.float32),
                v_norm=z(rows, torch.float32), cap=cap, page=page, table=table)


def _fill(c, tab, s, g):
    """Codes as the rotated coordinates of real keys and values give them (near Gaussian), norms near 1."""
    cap, B, H = s["cap"], c["B"], c["H"]
    for b in range(B):
        for h in range(H):
            width = tab["width"][h]
            pos = torch.arange(cap, device="cuda").view(1, 1, -1)
            one = dict(s, table=None if s["table"] is None else s["table"][b : b + 1])
            slot = (_slots(one, 1, H, pos.expand(1, H, -1))[0, h] if s["table"] is not None else (b * H + h) * cap + pos.view(-1))
            u = torch.randn((D, cap), device="cuda", generator=g)
            kc = torch.searchsorted(tab["thr"][width].contiguous(), u, right=True).t() * (width > 0)
            s["k_codes"].view(-1, 16 * c["bk"])[slot] = _pack(kc, tab["bit"][h], 4 * c["bk"])
            u = torch.randn((cap // 2, 2, D), device="cuda", generator=g)
            vc = torch.bucketize(u, tab["thr"][c["bv"]][: 2 ** c["bv"] - 1].contiguous(), right=True)
            s["v_codes"].view(-1, 32 * c["bv"])[slot[::2] >> 1] = _pack(vc.reshape(cap // 2, 2 * D), tab["vbit"].reshape(-1), 8 * c["bv"])
    s["k_norm"].copy_((0.2 * torch.randn(s["k_norm"].shape, device="cuda", generator=g)).exp())
    s["v_norm"].copy_((0.2 * torch.randn(s["v_norm"].shape, device="cuda", generator=g)).exp())


def _rows(c, sigma, shape, g):
    """Keys (or queries) [B, H, ..., 128] with each RoPE block's spread."""
    s = torch.cat([sigma, sigma], dim=-1).view(1, c["H"], *[1] * (len(shape) - 3), D)
    return torch.randn(shape, device="cuda", generator=g) * s


def _queries(c, sigma, rows, g):
    """Queries [B, H*G, rows.., 128] fp16 whose logits spread by about 2, as trained heads' do."""
    q = _rows(c, sigma, (c["B"], c["H"], c["G"], *rows, D), g)
    spread = (2 * sigma.double().pow(4).sum(-1)).sqrt().float() / math.sqrt(D)
    q = q * (2.0 / spread).view(1, -1, 1, *[1] * len(rows), 1)
    return q.view(c["B"], c["H"] * c["G"], *rows, D).half()


def _own_cache(plan, c, s):
    """The framework's cache object over the same records."""
    import rope_aware_quantized_gb300 as bg

    cache = bg.Cache(plan, c["B"], s["cap"], page_tokens=s["page"])
    for name in ("k_codes", "v_codes", "k_norm", "v_norm"):
        getattr(cache, name).copy_(s[name])
    if s["table"] is not None:
        cache.page_table.copy_(s["table"])
    return cache


def prepare(case, seed):
    c, g = dict(case), _generator(seed)
    st = dict(c=c)
    if c["op"] == "score_prefill":
        sigma = torch.tensor(np.stack([_sigma(h) for h in range(c["H"])]), dtype=torch.float32, device="cuda")
        st["q"] = _queries(c, sigma, (c["T"],), g)
        st["k"] = _rows(c, sigma, (c["B"], c["H"], c["T"], D), g).half()
        st["lse"] = torch.zeros(c["B"], c["H"] * c["G"], c["T"], device="cuda")
        rows, qk = c["T"] - c["row0"], st["q"].view(c["B"], c["H"], c["G"], c["T"], D)
        for r0 in range(c["row0"], c["T"], 1024):
            r1 = min(c["T"], r0 + 1024)
            s = torch.einsum("bhgrd,bhtd->bhgrt", qk[:, :, :, r0:r1].float(), st["k"].float()) / math.sqrt(D)
            seen = _visible(torch.arange(r0, r1, device="cuda").view(-1, 1), torch.arange(c["T"], device="cuda"), c["sinks"], c["window"])
            st["lse"][:, :, r0:r1] = s.masked_fill(~seen, -math.inf).logsumexp(-1).view(c["B"], -1, r1 - r0)
        st["scores"] = torch.zeros(c["B"], c["H"], c["T"], device="cuda")
        if own:  # the plan and the workspace that a user's program keeps
            import rope_aware_quantized_gb300 as bg

            st["plan"] = _plan(c["H"], c["G"], 3, 3)
            st["ws"] = torch.zeros(bg.bgtq_prefill_score_workspace(st["plan"], c["B"], c["T"], c["row0"]), dtype=torch.uint8, device="cuda")
        return st
    tab = _device_tables(c["H"], c["bk"], c["bv"])
    if c["op"] == "window_prefill":
        st["q"] = _queries(c, tab["sigma"], (c["T"],), g)
        st["k"] = _rows(c, tab["sigma"], (c["B"], c["H"], c["T"], D), g).half()
        st["v"] = torch.randn((c["B"], c["H"], c["T"], D), device="cuda", generator=g).half()
        st["cache"] = _cache(c, g, c["T"] + c["T"] % 2, 0)
        st["out"] = torch.zeros_like(st["q"])
        st["lse"] = torch.zeros(c["B"], c["H"] * c["G"], c["T"], device="cuda")
        if own:
            st["plan"] = _plan(c["H"], c["G"], c["bk"], c["bv"])
            st["own_cache"] = _own_cache(st["plan"], c, st["cache"])
        return st
    st["lens"] = _lens(c, g)
    st["cache"] = _cache(c, g, c["cap"], c["page"])
    _fill(c, tab, st["cache"], g)
    if c["op"] == "evict":
        # weights that a few positions gather most of, some of them equal, some never seen
        shape = (c["B"], c["H"], c["cap"])
        x = torch.exp(2.0 * torch.randn(shape, device="cuda", generator=g)).half().float()
        st["scores"] = torch.where(torch.rand(shape, device="cuda", generator=g) < 0.1, torch.zeros_like(x), x)
        page = c["page"]
        cap = -(-c["keep"] // page) * page if page else c["keep"] + c["keep"] % 2
        st["dst"] = _cache(c, g, cap, page)
        st["dst_scores"] = torch.zeros(c["B"], c["H"], cap, device="cuda")
        st["dst_lens"] = torch.zeros(c["B"], dtype=torch.int32, device="cuda")
        st["kept"] = torch.full((c["B"], c["H"], c["keep"]), -1, dtype=torch.int32, device="cuda")
        if own:
            st["plan"] = _plan(c["H"], 1, c["bk"], c["bv"])
            st["own_cache"], st["own_dst"] = _own_cache(st["plan"], c, st["cache"]), _own_cache(st["plan"], c, st["dst"])
        return st
    st["q"] = _queries(c, tab["sigma"], (), g)
    st["k_new"] = _rows(c, tab["sigma"], (c["B"], c["H"], D), g).half()
    st["v_new"] = torch.randn((c["B"], c["H"], D), device="cuda", generator=g).half()
    st["pos_new"] = st["lens"] - 1
    st["out"] = torch.zeros(c["B"], c["H"] * c["G"], D, dtype=torch.float16 if c["half"] else torch.float32, device="cuda")
    if c["op"] == "score_decode":
        st["scores_in"] = torch.rand((c["B"], c["H"], c["cap"]), device="cuda", generator=g)
        st["scores_out"] = torch.zeros_like(st["scores_in"])
    if own:
        import rope_aware_quantized_gb300 as bg

        st["plan"] = _plan(c["H"], c["G"], c["bk"], c["bv"])
        st["own_cache"] = _own_cache(st["plan"], c, st["cache"])
        n = (bg.bgtq_decode_window_workspace(st["plan"], c["B"], c["len_hi"], c["sinks"], c["window"]) if c["op"] == "window_decode"
             else bg.bgtq_decode_score_workspace(st["plan"], c["B"], c["len_hi"]))
        st["ws"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
    return st


# ----------------------------------------------------------------- the calls


def run(st):
    c = st["c"]
    if own:
        return _run_own(c, st)
    return {"window_decode": _window_decode, "window_prefill": _window_prefill, "score_decode": _score_decode,
            "score_prefill": _score_prefill, "evict": _evict}[c["op"]](c, st)


def _records(cache, get):
    return {n: get(cache, n) for n in ("k_codes", "v_codes", "k_norm", "v_norm")}


def _run_own(c, st):
    import rope_aware_quantized_gb300 as bg

    if c["op"] == "window_prefill":
        bg.bgtq_prefill_window_attn(st["plan"], st["q"], st["k"], st["v"], st["own_cache"], c["sinks"], c["window"], st["out"], lse=st["lse"])
        return dict(out=st["out"], lse=st["lse"], **_records(st["own_cache"], getattr))
    if c["op"] == "score_prefill":
        bg.bgtq_prefill_score(st["plan"], st["q"], st["k"], st["lse"], st["scores"], st["ws"], row0=c["row0"], sinks=c["sinks"], window=c["window"])
        return dict(scores=st["scores"])
    if c["op"] == "evict":
        bg.bgtq_evict(st["plan"], st["own_cache"], st["scores"], st["lens"], c["len_hi"], c["keep"], c["sinks"], c["recent"],
                      st["own_dst"], st["dst_scores"], st["dst_lens"], st["kept"])
        return dict(scores=st["dst_scores"], lens=st["dst_lens"], kept=st["kept"], **_records(st["own_dst"], getattr))
    new = dict(k_new=st["k_new"], v_new=st["v_new"], pos_new=st["pos_new"]) if c["step"] else {}
    if c["op"] == "window_decode":
        bg.bgtq_decode_window_attn(st["plan"], st["q"], st["own_cache"], st["lens"], c["len_hi"], c["sinks"], c["window"], st["out"],
                                   st["ws"], **new)
        got = dict(out=st["out"])
    else:
        bg.bgtq_decode_score_attn(st["plan"], st["q"], st["own_cache"], st["lens"], c["len_hi"], st["scores_in"], st["scores_out"],
                                  st["out"], st["ws"], **new)
        got = dict(out=st["out"], scores=st["scores_out"])
    return dict(got, **_records(st["own_cache"], getattr)) if c["step"] else got


# ----------------------------------------------------------------- plain forms


def _visible(i, j, sinks, window):
    """Whether the row at position i sees position j."""
    return (j <= i) & ((j < sinks) | (j > i - window))


def _softmax(s, seen):
    """Weights of masked logits in 32 bits; a row that sees nothing gives zeros."""
    s = s.masked_fill(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isfinite(m), m, torch.zeros_like(m)))
    return p / p.sum(-1, keepdim=True).clamp_min(1e-30)


def _weights(c, st, k, seen):
    q = st["q"].float().view(c["B"], c["H"], c["G"], D)
    return _softmax((q @ k.transpose(-1, -2)) * (1 / math.sqrt(D)), seen.unsqueeze(2))


def _step(c, tab, st):
    if c["step"]:
        _append(c, tab, st["cache"], st["k_new"], st["v_new"], st["pos_new"])


def _window_decode(c, st):
    tab = _device_tables(c["H"], c["bk"], c["bv"])
    _step(c, tab, st)
    n = st["lens"].to(torch.int64).view(-1, 1, 1)
    lo = (n - c["window"]).clamp_min(0)
    sink = torch.arange(min(c["sinks"], c["cap"]), device="cuda").view(1, 1, -1).expand(c["B"], 1, -1)
    win = n - 1 - torch.arange(min(c["window"], c["len_hi"]), device="cuda").view(1, 1, -1)
    pos = torch.cat([sink, win], -1).expand(-1, c["H"], -1)
    seen = torch.cat([(sink < lo) & (sink < n), win >= 0], -1).expand(-1, c["H"], -1)
    k, v = _dequant(c, tab, st["cache"], pos.clamp_min(0))
    out = _weights(c, st, k, seen) @ v
    out = out.view(st["out"].shape).to(st["out"].dtype)
    got = dict(out=out)
    return dict(got, **_records(st["cache"], dict.get)) if c["step"] else got


def _window_prefill(c, st):
    B, H, G, T, W = c["B"], c["H"], c["G"], c["T"], c["window"]
    tab = _device_tables(H, c["bk"], c["bv"])
    # blocks of W rows: block n sees the sinks and the positions of blocks n - 1 and n
    nb, S = -(-T // W), min(c["sinks"], T)
    pad = lambda x, lo: torch.nn.functional.pad(x.float(), (0, 0, lo, nb * W - T))  # noqa: E731
    q = pad(st["q"], 0).view(B, H, G, nb, W, D)
    band = lambda x: torch.cat([pad(x, W)[:, :, : nb * W].view(B, H, nb, W, D), pad(x, 0).view(B, H, nb, W, D)], 3)  # noqa: E731
    sinks = lambda x: x[:, :, :S].float().unsqueeze(2).expand(B, H, nb, S, D)  # noqa: E731
    keys = torch.cat([sinks(st["k"]), band(st["k"])], 3)
    vals = torch.cat([sinks(st["v"]), band(st["v"])], 3)
    start = (torch.arange(nb, device="cuda") * W).view(nb, 1, 1)
    i = start + torch.arange(W, device="cuda").view(1, W, 1)
    js = torch.arange(S, device="cuda").view(1, 1, S)
    jb = start - W + torch.arange(2 * W, device="cuda").view(1, 1, 2 * W)
    # a sink inside the band counts there; a band position is at most the row
    seen = torch.cat([(js <= i) & (js < start - W), (jb >= 0) & (jb < T) & _visible(i, jb, S, W)], 2)
    s = torch.einsum("bhgnid,bhnjd->bhgnij", q, keys).mul_(1 / math.sqrt(D)).masked_fill_(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    out = torch.einsum("bhgnij,bhnjd->bhgnid", p, vals) / l.clamp_min(1e-30)
    out = out.reshape(B, H * G, nb * W, D)[:, :, :T].half()
    lse = (m + l.log()).reshape(B, H * G, nb * W)[:, :, :T]
    cache, Te = st["cache"], T + T % 2
    kc, kr, vc, vr = _encode_kv(c, tab, st["k"], st["v"])
    even = lambda x: torch.nn.functional.pad(x, (0, 0, 0, Te - T))  # noqa: E731
    cache["k_codes"].view(B, H, Te, -1)[:, :, :T] = _pack(kc, tab["bit"].view(1, H, 1, D), 4 * c["bk"])
    cache["v_codes"].copy_(_pack(even(vc).reshape(B, H, Te // 2, 2 * D), tab["vbit"].reshape(-1), 8 * c["bv"]).reshape(-1))
    cache["k_norm"].view(B, H, Te)[:, :, :T] = kr
    cache["v_norm"].view(B, H, Te)[:, :, :T] = vr
    return dict(out=out, lse=lse, **_records(cache, dict.get))


def _score_decode(c, st):
    tab = _device_tables(c["H"], c["bk"], c["bv"])
    _step(c, tab, st)
    pos = torch.arange(c["len_hi"], device="cuda").view(1, 1, -1).expand(c["B"], c["H"], -1)
    seen = pos < st["lens"].view(-1, 1, 1)
    k, v = _dequant(c, tab, st["cache"], pos)
    p = _weights(c, st, k, seen)
    out = (p @ v).view(st["out"].shape).to(st["out"].dtype)
    before = st["scores_in"][:, :, : c["len_hi"]]
    if c["step"]:  # a new position has no weight yet
        before = before.masked_fill(pos == st["pos_new"].view(-1, 1, 1), 0.0)
    scores = st["scores_out"]
    scores[:, :, : c["len_hi"]] = torch.where(seen, before + p.sum(2), scores[:, :, : c["len_hi"]])
    got = dict(out=out, scores=scores)
    return dict(got, **_records(st["cache"], dict.get)) if c["step"] else got


def _score_prefill(c, st):
    B, H, G, T, r0 = c["B"], c["H"], c["G"], c["T"], c["row0"]
    q = st["q"].view(B, H, G, T, D)[:, :, :, r0:].reshape(B, H, G * (T - r0), D).float()
    lse = st["lse"].view(B, H, G, T)[:, :, :, r0:].reshape(B, H, G * (T - r0), 1)
    i = torch.arange(r0, T, device="cuda").repeat(G).view(-1, 1)
    seen = _visible(i, torch.arange(T, device="cuda"), c["sinks"], c["window"])
    s = torch.matmul(q, st["k"].float().transpose(-1, -2)).mul_(1 / math.sqrt(D)).sub_(lse).masked_fill_(~seen, -math.inf)
    return dict(scores=s.exp_().sum(2))


def _evict(c, st):
    B, H, N, K = c["B"], c["H"], c["len_hi"], c["keep"]
    n = st["lens"].to(torch.int64).view(B, 1, 1)
    pos = torch.arange(N, device="cuda").view(1, 1, N)
    x = st["scores"][:, :, :N]
    always = (pos < c["sinks"]) | (pos >= n - c["recent"])
    x = x.masked_fill(always, math.inf).masked_fill((pos >= n).expand(B, H, N), -math.inf)
    best = x.sort(dim=-1, descending=True, stable=True).indices[:, :, : min(K, N)]
    m = n.clamp_max(K)
    best = torch.where(torch.arange(best.shape[-1], device="cuda") < m, best, torch.full_like(best, N)).sort(-1).values
    valid = best < N
    src, dst = st["cache"], st["dst"]
    at = torch.where(valid, best, torch.zeros_like(best))
    to = torch.arange(best.shape[-1], device="cuda").view(1, 1, -1).expand_as(best)
    fs, ts = _slots(src, B, H, at), _slots(dst, B, H, to)
    put = lambda name, w, f, t, ok: dst[name].view(-1, w).index_put_((t[ok],), src[name].view(-1, w)[f[ok]])  # noqa: E731
    put("k_codes", 16 * c["bk"], fs, ts, valid)
    put("k_norm", 1, fs, ts, valid)
    put("v_norm", 1, fs, ts, valid)
    # values: every token's codes out of its pair record, into its half of the new one
    width = torch.tensor(c["bv"], device="cuda")
    bits = _device_tables(H, c["bk"], c["bv"])["vbit"]
    codes = _fields(_words(src["v_codes"].view(-1, 32 * c["bv"])[fs >> 1]), bits[fs & 1], width)
    codes = torch.nn.functional.pad(codes * valid.unsqueeze(-1), (0, 0, 0, best.shape[-1] % 2))
    rec = _pack(codes.reshape(B, H, -1, 2 * D), bits.reshape(-1), 8 * c["bv"])
    first = valid[:, :, ::2]
    dst["v_codes"].view(-1, 32 * c["bv"]).index_put_((ts[:, :, ::2][first] >> 1,), rec[first])
    k = best.shape[-1]
    st["kept"][:, :, :k] = torch.where(valid, best, torch.full_like(best, -1)).to(torch.int32)
    st["dst_scores"][:, :, :k] = torch.where(valid, st["scores"].gather(2, at), st["dst_scores"][:, :, :k])
    st["dst_lens"].copy_(m.view(-1))
    return dict(scores=st["dst_scores"], lens=st["dst_lens"], kept=st["kept"], **_records(dst, dict.get))


# ----------------------------------------------------------------- the floors


def _expected(c, most=None):
    """Positions of all sequences together (the first is the longest, the others uniform), each at most `most`."""
    mean = (c["len_lo"] + c["len_hi"]) / 2
    if most is None or most >= c["len_hi"]:
        return c["len_hi"] + (c["B"] - 1) * mean
    if c["len_hi"] == c["len_lo"]:
        return c["B"] * min(most, c["len_hi"])
    lo, hi = c["len_lo"], c["len_hi"]
    below = (min(hi, max(lo, most)) - lo) / (hi - lo)
    return min(most, hi) + (c["B"] - 1) * (below * (lo + min(hi, max(lo, most))) / 2 + (1 - below) * most)


def work(case):
    c = case
    if c["op"] == "evict":
        n, kept = _expected(c), _expected(c, c["keep"])
        rec = 16 * c["bk"] + 16 * c["bv"] + 8 + 4
        return dict(bytes=c["H"] * (4 * n + kept * (2 * rec + 4)), flops=c["H"] * n)
    hq = c["H"] * c["G"]
    if c["op"] in ("window_prefill", "score_prefill"):
        T, W, S = c["T"], c["window"], c["sinks"]
        i = np.arange(c.get("row0", 0), T, dtype=np.float64)
        seen = np.minimum(i + 1, W) + np.minimum(S, np.maximum(i + 1 - W, 0))
        pairs, rows = c["B"] * hq * float(seen.sum()), len(i)
        if c["op"] == "window_prefill":
            byts = c["B"] * T * (hq * (2 * 256 + 4) + c["H"] * (512 + 16 * c["bk"] + 16 * c["bv"] + 8))
            return dict(bytes=byts, flops=4 * D * pairs)
        return dict(bytes=c["B"] * (rows * hq * 260 + c["H"] * T * 260), flops=2 * D * pairs)
    rec = 16 * c["bk"] + 16 * c["bv"] + 8
    n = _expected(c, c["sinks"] + c["window"] if c["op"] == "window_decode" else None)
    byts = c["H"] * n * (rec + (8 if c["op"] == "score_decode" else 0)) + c["B"] * hq * D * (2 + (2 if c["half"] else 4))
    byts += c["B"] * c["H"] * (512 + rec) if c["step"] else 0
    return dict(bytes=byts, flops=4 * D * c["G"] * c["H"] * n)


# ----------------------------------------------------------------- 64 bits


def _bits_of(rec):
    return ((rec.unsqueeze(-1) >> torch.arange(8, dtype=torch.uint8, device=rec.device)) & 1).flatten(-2)


def _rows64(c, s, b, h, pos):
    """Keys and values of positions pos [N] of one (sequence, head) in 64 bits, from the records' single bits and plain butterflies."""
    _, t = _tables(c["H"], c["bk"], c["bv"])
    cent = torch.tensor(_codebooks()[0], device="cuda")
    if s["table"] is None:
        slot = (b * c["H"] + h) * s["cap"] + pos
    else:
        slot = (s["table"][b, pos // s["page"]].long() * c["H"] + h) * s["page"] + pos % s["page"]
    kb = _bits_of(s["k_codes"].view(-1, 16 * c["bk"])[slot])
    y = torch.zeros(len(pos), D, dtype=torch.float64, device="cuda")
    for j in range(int(t["n"][h])):
        w, at = int(t["width"][h][j]), int(t["bit"][h][j])
        y[:, j] = cent[w][(kb[:, at : at + w].long() << torch.arange(w, device="cuda")).sum(-1)]
    j = 0
    k = torch.zeros_like(y)
    while j < t["n"][h]:
        p = int(t["piece"][h][j])
        x = _walsh64(y[:, j : j + p])
        f = torch.tensor(t["sk"][h][j : j + p] * t["dewhite"][h][j : j + p] / math.sqrt(p), device="cuda")
        k[:, t["perm"][h][j : j + p].tolist()] = x * f
        j += p
    vb = _bits_of(s["v_codes"].view(-1, 32 * c["bv"])[slot >> 1]).view(len(pos), D, 2, c["bv"])
    vb = vb.gather(2, (slot & 1).view(-1, 1, 1, 1).expand(-1, D, 1, c["bv"])).squeeze(2).long()
    v = _walsh64(cent[c["bv"]][(vb << torch.arange(c["bv"], device="cuda")).sum(-1)])
    v = v * torch.tensor(t["sv"][h] / math.sqrt(D), device="cuda")
    return k * s["k_norm"][slot].double().unsqueeze(-1), v * s["v_norm"][slot].double().unsqueeze(-1)


def _walsh64(x):
    n = x.shape[-1]
    h = 1
    while h < n:
        x = x.reshape(x.shape[0], -1, 2, h)
        x = torch.stack([x[:, :, 0] + x[:, :, 1], x[:, :, 0] - x[:, :, 1]], 2).reshape(x.shape[0], n)
        h *= 2
    return x


def exact(case, seed):
    c, st = case, prepare(case, seed)
    if c["op"] == "evict":
        return None  # moves records and picks whole numbers: nothing is computed in floating point
    B, H, G = c["B"], c["H"], c["G"]
    nothing = dict.fromkeys(("k_codes", "v_codes", "k_norm", "v_norm"))
    if c["op"] == "score_prefill":
        T = c["T"]
        pairs = B * H * G * (T - c["row0"]) * T
        if pairs > 6e9:
            return None
        total = torch.zeros(B, H, T, dtype=torch.float64, device="cuda")
        at = torch.arange(T, device="cuda")
        for b in range(B):
            for hq in range(H * G):
                k = st["k"][b, hq // G].double()
                for r0 in range(c["row0"], T, 4096):
                    r = torch.arange(r0, min(T, r0 + 4096), device="cuda")
                    s = st["q"][b, hq, r].double() @ k.T / math.sqrt(D) - st["lse"][b, hq, r].double().unsqueeze(1)
                    out = (at > r.unsqueeze(1)) | ((at <= r.unsqueeze(1) - c["window"]) & (at >= c["sinks"]))
                    total[b, hq // G] += torch.where(out, torch.zeros_like(s), s.exp()).sum(0)
        return dict(scores=total)
    if c["op"] == "window_prefill":
        T, W, S = c["T"], c["window"], min(c["sinks"], c["T"])
        out = torch.zeros(B, H * G, T, D, dtype=torch.float64, device="cuda")
        lse = torch.zeros(B, H * G, T, dtype=torch.float64, device="cuda")
        for b in range(B):
            for hq in range(H * G):
                k, v = st["k"][b, hq // G].double(), st["v"][b, hq // G].double()
                for r0 in range(0, T, 1024):
                    r = torch.arange(r0, min(T, r0 + 1024), device="cuda")
                    lo = max(0, r0 - W + 1)
                    at = torch.cat([torch.arange(min(S, lo), device="cuda"), torch.arange(lo, int(r[-1]) + 1, device="cuda")])
                    s = st["q"][b, hq, r].double() @ k[at].T / math.sqrt(D)
                    gap = r.unsqueeze(1) - at
                    s = torch.where((gap >= 0) & ((gap < W) | (at < S)), s, torch.full_like(s, -math.inf))
                    lse[b, hq, r] = s.logsumexp(-1)
                    out[b, hq, r] = s.softmax(-1) @ v[at]
        return dict(nothing, out=out, lse=lse)
    tab = _device_tables(H, c["bk"], c["bv"])
    _step(c, tab, st)  # the records' bytes are whole numbers of the format
    out = torch.zeros(B, H * G, D, dtype=torch.float64, device="cuda")
    scores = st["scores_out"].double() if c["op"] == "score_decode" else None
    for b in range(B):
        n = int(st["lens"][b])
        pos = torch.arange(n, device="cuda")
        if c["op"] == "window_decode":
            pos = pos[(pos < c["sinks"]) | (pos >= n - c["window"])]
        for h in range(H):
            k, v = _rows64(c, st["cache"], b, h, pos)
            p = (st["q"][b, h * G : (h + 1) * G].double() @ k.T / math.sqrt(D)).softmax(-1)
            out[b, h * G : (h + 1) * G] = p @ v
            if scores is not None:
                was = st["scores_in"][b, h, :n].double()
                if c["step"]:
                    was[int(st["pos_new"][b])] = 0.0
                scores[b, h, :n] = was + p.sum(0)
    got = dict(out=out) if scores is None else dict(out=out, scores=scores)
    return dict(nothing, **got) if c["step"] else got
