"""Pins of the oracle's bounded-cache functions (readings R23-R25)."""

import numpy as np
import pytest

from oracle import bgtq_oracle as O


def test_visible_positions():
    assert list(O.decode_visible(10, 2, 3)) == [0, 1, 7, 8, 9]
    assert list(O.decode_visible(4, 2, 3)) == [0, 1, 2, 3]
    assert list(O.decode_visible(10, 0, 1)) == [9]
    assert list(O.decode_visible(3, 7, 1)) == [0, 1, 2]
    assert list(O.decode_visible(0, 2, 3)) == []
    i, j = np.arange(5)[:, None], np.arange(5)[None, :]
    assert np.array_equal(O.visible(i, j, 0, 5), j <= i)  # a window as long as the sequence: causal
    assert O.visible(i, j, 1, 2).sum(axis=1).tolist() == [1, 2, 3, 3, 3]


def test_weights_and_window_prefill_agree_with_the_pinned_attention():
    r = np.random.default_rng(0)
    q, k, v = (r.standard_normal((2, 6, 128)).astype(np.float16), r.standard_normal((6, 128)).astype(np.float16),
               r.standard_normal((6, 128)).astype(np.float16))
    out, lse, w = O.prefill_window(q, k, v, 0, 6)
    assert np.abs(out - O.prefill_attention(q, k, v)).max() < 1e-13  # no window: reading R21
    assert np.abs(w.sum(axis=2) - 1).max() < 1e-14
    out, lse, w = O.prefill_window(q, k, v, 1, 2)
    for i in range(6):
        at = O.decode_visible(i + 1, 1, 2)
        assert np.abs(out[:, i] - O.attention(q[:, i], k[at], v[at])).max() < 1e-13
        assert np.abs(w[:, i][:, at] - O.attention_weights(q[:, i], k[at])).max() < 1e-14
        assert w[:, i].sum() == pytest.approx(2)
        s = q[:, i].astype(np.float64) @ k[at].T.astype(np.float64) / np.sqrt(128)
        assert np.abs(np.exp(s - lse[:, i:i + 1]).sum(axis=1) - 1).max() < 1e-13


@pytest.mark.parametrize("scores,n,keep,sinks,recent,want", [
    ([5, 1, 4, 2, 3], 5, 3, 0, 0, [0, 2, 4]),
    ([1, 1, 1, 1, 1], 5, 3, 0, 0, [0, 1, 2]),                 # ties: the lower position
    ([0, 9, 9, 9, 0], 5, 3, 1, 1, [0, 1, 4]),
    ([0.0, -0.0, np.nan, -np.inf, np.inf], 5, 3, 0, 0, [0, 1, 4]),
    ([np.nan, -np.inf, np.nan, -1.0, np.nan], 5, 3, 0, 0, [0, 1, 3]),
    ([3, 2, 1], 3, 5, 1, 1, [0, 1, 2]),                       # shorter than the budget
    ([3, 2, 9, 1], 4, 2, 1, 1, [0, 3]),                       # the sinks and the recent ones fill it
    ([], 0, 2, 0, 0, []),
])
def test_evict_positions(scores, n, keep, sinks, recent, want):
    assert O.evict_positions(np.array(scores), n, keep, sinks, recent).tolist() == want
