"""CPU oracle of the rotary operators and of the 4-bit cache, from their
definitions: rotation of 2-D blocks in float32 (one rounding an operation),
blocks of 16 values of e2m1 under a scale of 5 exponent and 3 mantissa bits, the
byte layout of a group of 16 positions, and attention in float64."""

import numpy as np

D = 128
GROUP_BYTES = 2304
LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def rope_table(inv_freq, n_pos, scale=1.0):
    a = np.arange(n_pos, dtype=np.float64)[:, None] * np.asarray(inv_freq, np.float64)[None, :]
    return (scale * np.cos(a)).astype(np.float32), (scale * np.sin(a)).astype(np.float32)


def rope(x, cos, sin, pos, layout=0, axis=None, inverse=False, exact=False):
    """Rows x [..., T, 128]; pos [axes][..., T] (broadcast against x's rows); float32 operations, or with `exact` float64."""
    axis = np.zeros(64, np.int64) if axis is None else np.asarray(axis)
    ty = np.float64 if exact else np.float32
    c = np.stack([cos[pos[axis[i]], i] for i in range(64)], -1).astype(ty)
    s = np.stack([sin[pos[axis[i]], i] for i in range(64)], -1).astype(ty)
    s = -s if inverse else s
    x = x.astype(ty)
    lo, hi = (x[..., :64], x[..., 64:]) if layout == 0 else (x[..., 0::2], x[..., 1::2])
    a, b = lo * c - hi * s, hi * c + lo * s
    out = np.empty(np.broadcast_shapes(x.shape, a.shape[:-1] + (D,)), ty)
    if layout == 0:
        out[..., :64], out[..., 64:] = a, b
    else:
        out[..., 0::2], out[..., 1::2] = a, b
    return out


def scale_value(byte):
    """The number of a scale byte: 5 exponent bits (bias 15) and 3 mantissa bits."""
    b = np.asarray(byte, np.int64)
    e, m = b >> 3, b & 7
    return np.where(e == 0, m * 2.0 ** -17, (8 + m) * 2.0 ** (e - 18.0))


def scale_byte(amax):
    """amax / 6 to the nearest scale, ties to the even byte, at most 10240."""
    table = scale_value(np.arange(227))
    y = np.asarray(amax, np.float64) / 6
    hi = np.clip(np.searchsorted(table, y), 0, 226)  # first scale >= y
    lo = np.maximum(hi - 1, 0)
    down, up = y - table[lo], table[hi] - y
    # (y is amax / 6 rounded to 64 bits: a tie is exact, or it is none)
    return np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi).astype(np.uint8)


def fp4_encode(x):
    """Rows x [..., 128] of fp16 -> codes uint8 [..., 128], scale bytes uint8 [..., 8]."""
    x = np.asarray(x, np.float64)
    blocks = x.reshape(*x.shape[:-1], 8, 16)
    byte = scale_byte(np.abs(blocks).max(-1))
    s = scale_value(byte)[..., None]
    a = np.abs(blocks)
    dist = np.abs(a[..., None] - LEVELS * s[..., None])  # exact: few bits each
    mag = dist.argmin(-1)
    tie = (mag < 7) & (np.take_along_axis(dist, np.minimum(mag + 1, 7)[..., None], -1)[..., 0] == dist.min(-1)) & (mag % 2 == 1)
    mag = np.where(s > 0, np.where(tie, mag + 1, mag), 0)
    return (mag + 8 * np.signbit(blocks)).astype(np.uint8).reshape(x.shape), byte


def fp4_value(codes, byte):
    v = np.where(codes & 8, -1.0, 1.0) * LEVELS[codes & 7]
    return (v.reshape(*v.shape[:-1], 8, 16) * scale_value(byte)[..., None]).reshape(v.shape)


def _index():
    p, d = np.meshgrid(np.arange(16), np.arange(D), indexing="ij")
    k = 64 * p + 16 * (d // 4 % 4) + 2 * (d // 16) + d // 2 % 2
    v = 1024 + 512 * (d // 64) + 64 * (d % 8) + 16 * (p // 2 % 4) + 4 * (d // 16 % 4) + 2 * (p // 8) + d // 8 % 2
    p8, b8 = np.meshgrid(np.arange(16), np.arange(8), indexing="ij")
    return k, d % 2, v, p % 2, 2048 + 8 * p8 + b8, 2176 + 32 * (p8 // 2 % 4) + 4 * b8 + 2 * (p8 // 8) + p8 % 2


KB, KN, VB, VN, KS, VS = _index()


def write(group, p, kc, ks, vc, vs):
    """Position p of a group (uint8 [2304], changed in place) from its codes and scale bytes."""
    for at, nib, code in ((KB[p], KN[p], kc), (VB[p], VN[p], vc)):
        for i in range(D):
            sh = 4 * int(nib[i])
            group[at[i]] = (int(group[at[i]]) & ~(15 << sh) & 255) | int(code[i]) << sh
    group[KS[p]], group[VS[p]] = ks, vs


def read(groups):
    """Groups [..., 2304] -> codes and scale bytes of keys and values, [..., 16, 128] and [..., 16, 8]."""
    nib = lambda at, n: (groups[..., at] >> (4 * n).astype(np.uint8)) & 15  # noqa: E731
    return nib(KB, KN), groups[..., KS], nib(VB, VN), groups[..., VS]


def attention(q, k, first, scale):
    """Weights [T][n] of rows q [T][128] at positions first .. over keys k [n][128], float64; a row before position 0: zeros."""
    q, k = np.asarray(q, np.float64), np.asarray(k, np.float64)
    s = scale * q @ k.T
    seen = np.arange(len(k))[None, :] <= first + np.arange(len(q))[:, None]
    s = np.where(seen, s, -np.inf)
    m = np.where(seen.any(-1), s.max(-1, initial=-np.inf), 0.0)[:, None]
    w = np.exp(s - m)
    return w / np.maximum(w.sum(-1, keepdims=True), 1e-300)
