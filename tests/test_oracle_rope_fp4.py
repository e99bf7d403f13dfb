"""The oracle of the rotary operators and of the 4-bit cache against hand-worked values."""

import numpy as np
import pytest

from oracle import rope_fp4_oracle as F


@pytest.mark.parametrize("layout", [0, 1])
def test_rotation_of_one_block(layout):
    cos, sin = F.rope_table([np.pi / 2] * 64, 4)
    x = np.zeros((1, 128), np.float16)
    lo, hi = (5, 69) if layout == 0 else (10, 11)
    x[0, lo], x[0, hi] = 3, 4
    y = F.rope(x, cos, sin, np.array([[1]]), layout)  # a quarter turn: (3, 4) -> (-4, 3)
    assert np.allclose(y[0, [lo, hi]], [-4, 3], atol=1e-6)
    z = F.rope(y, cos, sin, np.array([[1]]), layout, inverse=True)
    assert np.allclose(z, x, atol=1e-6)


def test_axes_choose_the_position():
    cos, sin = F.rope_table(np.linspace(0.1, 1, 64), 50)
    x = np.random.default_rng(0).standard_normal((3, 128)).astype(np.float16)
    pos = np.array([[3, 4, 5], [7, 8, 9]])
    axis = [0] * 32 + [1] * 32
    y = F.rope(x, cos, sin, pos, 0, axis)
    for a in range(2):
        z = F.rope(x, cos, sin, pos[a:a + 1])
        at = np.r_[32 * a:32 * a + 32, 64 + 32 * a:96 + 32 * a]
        assert np.array_equal(y[:, at], z[:, at])


def test_scales():
    assert F.scale_value(226) == 10240 and F.scale_value(8) == 2.0 ** -14 and F.scale_value(7) == 7 * 2.0 ** -17
    # the byte is bits 14..7 of the number in fp16
    b = np.arange(227)
    assert np.array_equal((b.astype(np.uint16) << 7).view(np.float16).astype(np.float64), F.scale_value(b))
    assert F.scale_byte(0.0) == 0 and F.scale_byte(65504.0) == 226
    assert np.array_equal(F.scale_byte(6 * F.scale_value(b)), b)
    assert F.scale_byte(6 * 2.0 ** -18) == 0  # a tie with 0
    mid = 3 * (F.scale_value(b[:-1]) + F.scale_value(b[1:]))
    assert np.array_equal(F.scale_byte(mid), b[:-1] + b[:-1] % 2)  # to the even byte


def test_codes_ties_and_signs():
    x = np.zeros(128)
    x[:16] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -5, 0.2503, -0.0, 0.0, 4.9, -6]  # scale 1
    codes, byte = F.fp4_encode(x.astype(np.float16))
    assert F.scale_value(byte[0]) == 1 and (byte[1:] == 0).all()
    assert codes[:16].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 8, 10, 14, 1, 8, 0, 6, 15]
    assert (codes[16:] == 0).all()


def test_group_bytes_are_each_written_once():
    for at, nib, lo, hi in ((F.KB, F.KN, 0, 1024), (F.VB, F.VN, 1024, 2048)):
        n = np.sort((2 * at + nib).reshape(-1))
        assert np.array_equal(n, np.arange(2 * lo, 2 * hi))
    assert np.array_equal(np.sort(np.r_[F.KS.reshape(-1), F.VS.reshape(-1)]), np.arange(2048, 2304))


def test_read_what_was_written():
    r = np.random.default_rng(1)
    g = r.integers(0, 256, F.GROUP_BYTES).astype(np.uint8)
    old = [a.copy() for a in F.read(g)]
    new = [r.integers(0, m, n).astype(np.uint8) for m, n in ((16, 128), (227, 8), (16, 128), (227, 8))]
    F.write(g, 5, *new)
    for a, b, c in zip(F.read(g), old, new):
        b[5] = c
        assert np.array_equal(a, b)


def test_values_are_exact_in_fp16_and_near():
    x = (np.random.default_rng(2).standard_normal((64, 128)) * 10.0 ** np.random.default_rng(3).uniform(-3, 4, (64, 1))).astype(np.float16)
    x = np.clip(x, -60000, 60000).astype(np.float16)
    v = F.fp4_value(*F.fp4_encode(x))
    assert np.array_equal(v, v.astype(np.float16).astype(np.float64))
    a = np.abs(x.astype(np.float64)).reshape(64, 8, 16).max(-1, keepdims=True)
    # a step is at most 2 (between 4 and 6) of a scale that is at most (1 + 2^-4) amax / 6, the
    # top code up to 2^-4 of amax short, and a scale below 2^-14 off by 2^-18
    tol = np.maximum(a * (1 + 2.0 ** -4) / 6 + 6 * 2.0 ** -18, a * 2.0 ** -3)
    assert (np.abs(v - x.astype(np.float64)).reshape(64, 8, 16) <= tol).all()


def test_attention_rows_before_the_start_give_zeros():
    r = np.random.default_rng(4)
    w = F.attention(r.standard_normal((4, 128)), r.standard_normal((2, 128)), -2, 0.1)
    assert (w[:2] == 0).all() and np.allclose(w[2], [1, 0]) and np.isclose(w[3].sum(), 1)
