"""Host checks of an eviction's buffers (no GPU: fake addresses, never
dereferenced): `kept`, `dst_scores` and `dst_lens` meet none of the buffers
that the call reads."""

import pytest

from tests.test_bounded_host import BASE, FAR, desc, evict

APART = dict(kept=FAR + (1 << 32), dst_scores=FAR + (2 << 32), dst_lens=FAR + (3 << 32))


@pytest.mark.parametrize("name", sorted(APART))
@pytest.mark.parametrize("at,frag", [
    (BASE, "overlaps"),                       # the source's k_codes, scores and seq_lens
    (BASE + (1 << 28), "k_norm"), (BASE + (2 << 28), "v_codes"), (BASE + (3 << 28), "v_norm"),
    (BASE + (2 << 28) + 2 * 128 * 48 - 4, "v_codes"),  # its last word
    (5 << 40, "scores"), (6 << 40, "seq_lens"),
])
def test_written_buffers_over_what_is_read(name, at, frag):
    rc, msg = evict(scores=5 << 40, lens=6 << 40, **{**APART, name: at})
    assert rc == -1 and "overlaps" in msg and frag in msg and msg.startswith(name), (rc, msg)


@pytest.mark.parametrize("name", sorted(APART))
def test_written_buffers_over_a_page_table(name):
    for which, word in (("src", "source"), ("dst", "destination")):
        kw = {"src": desc(page=16, table=7 << 40)} if which == "src" else {"dst": desc(FAR, 64, page=16, table=7 << 40)}
        rc, msg = evict(**{**APART, name: (7 << 40) + 8}, **kw)
        assert rc == -1 and f"{word}'s page table" in msg, (rc, msg)


def test_buffers_next_to_what_is_read():
    for at in (BASE + 2 * 128 * 48, BASE + (1 << 28) + 2 * 128 * 4, BASE + (2 << 28) + 2 * 128 * 48):
        for name in APART:
            assert "host-only" in evict(**{**APART, name: at})[1]
