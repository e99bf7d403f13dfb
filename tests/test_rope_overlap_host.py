"""Host checks of which outputs bgtq_rope_rows takes (no GPU, and none is used: every call below is
refused, one that is right so far by what is checked next)."""

import numpy as np
import pytest

from tests.test_rope_fp4_host import call_rows, rows

BASE, FAR = 1 << 30, 1 << 40
ELEM = {0: 2, 1: 4, 2: 2}


def own(q, qo, n, ext, din, dout):
    """Whether q_out is refused for its input (else the keys are, whose output lies 16 bytes into them)."""
    rc, msg = call_rows(q=q, qo=qo, nq=n, batch=ext[0], t=ext[1], din=din, dout=dout,
                        k=rows(FAR, 1 << 30, 1 << 20, 4096), ko=rows(FAR + 16, 1 << 30, 1 << 20, 4096), nk=1)
    assert rc == -1 and "_out overlaps" in msg, msg
    return "q_out overlaps q " in msg


def cross(qo, nq, ko, nk, ext, dout):
    """Whether q_out and k_out are refused for one another (else the queries are, 16 bytes into their output)."""
    rc, msg = call_rows(q=rows(qo.data + 16, qo.stride_b, qo.stride_h, qo.stride_t), qo=qo, nq=nq, batch=ext[0], t=ext[1], din=dout, dout=dout,
                        k=rows(FAR, 1 << 30, 1 << 20, 4096), ko=ko, nk=nk)
    assert rc == -1 and "overlap" in msg, msg
    return "q_out and k_out" in msg


def meet(a, na, b, nb, ext, ea, eb):
    """Whether any byte of the rows a is one of the rows b, row by row."""
    def at(r, n, e):
        return [r.data + e * (i * r.stride_b + h * r.stride_h + t * r.stride_t) for i in range(ext[0]) for h in range(n) for t in range(ext[1])]
    x, y = np.array(at(a, na, ea))[:, None], np.array(at(b, nb, eb))[None]
    return bool(((x < y + 128 * eb) & (y < x + 128 * ea)).any())


# a projection's output [B][T][12 heads][128] and, of a second layout, [B][12 heads][T][128]
LAYOUTS = [lambda ext: (ext[1] * 12 * 128, 128, 12 * 128), lambda ext: (12 * ext[1] * 128, ext[1] * 128, 128)]


@pytest.mark.parametrize("layout", LAYOUTS)
def test_rows_beside_their_input_are_taken(layout):
    """Queries rotated into other columns of the tensor that they come from; in place; and what meets."""
    ext = (2, 5)
    s = layout(ext)
    q = rows(BASE, *s)
    head = 2 * s[1]
    assert not own(q, rows(BASE + 4 * head, *s), 4, ext, 0, 0)
    assert not own(rows(BASE + 4 * head, *s), q, 4, ext, 0, 0)
    assert not own(q, q, 4, ext, 0, 0)
    assert not own(q, rows(BASE + 4 * head, *s), 4, ext, 0, 2)  # (another type of the same size, apart)
    assert own(q, q, 4, ext, 0, 2)
    assert own(q, rows(BASE + 3 * head, *s), 4, ext, 0, 0)
    assert own(q, rows(BASE + 16, *s), 4, ext, 0, 0)
    # strides that differ, in one another's extent: not looked into, refused
    assert own(q, rows(BASE + 4 * head, 4 * s[0], 4 * s[1], 4 * s[2]), 2, ext, 0, 0)


def test_the_check_is_exact_where_the_strides_agree():
    rng = np.random.default_rng(0)
    seen = []
    for _ in range(3000):
        ext, n = (int(rng.integers(1, 4)), int(rng.integers(1, 5))), int(rng.integers(1, 5))
        order, st, span = rng.permutation(3), [0, 0, 0], 128
        dims = (ext[0], n, ext[1])
        for i in order:
            st[i] = span + 64 * int(rng.integers(0, 8))
            span = st[i] * (dims[i] - 1) + span
        din, dout = [(0, 0), (1, 1), (0, 2), (2, 2)][int(rng.integers(0, 4))]
        a = rows(BASE, *st)
        far = 2 * span * ELEM[din]
        b = rows(BASE + 16 * int(rng.integers(-far // 16, far // 16)) if rng.random() < 0.9 else BASE, *st)
        want = meet(a, n, b, n, ext, ELEM[din], ELEM[dout]) and not (a.data == b.data and din == dout)
        assert own(a, b, n, ext, din, dout) == want, (ext, n, st, din, dout, b.data - BASE)
        seen.append(want)
    assert 500 < sum(seen) < 2500


def test_outputs_of_queries_and_keys_do_not_meet():
    """The queries' output and the keys': side by side in one tensor, or refused."""
    rng = np.random.default_rng(1)
    seen = []
    for _ in range(2000):
        ext, nq, nk = (int(rng.integers(1, 4)), int(rng.integers(1, 5))), int(rng.integers(1, 5)), int(rng.integers(1, 5))
        order, st, span = rng.permutation(3), [0, 0, 0], 128
        dims = (ext[0], nq + nk, ext[1])
        for i in order:
            st[i] = span + 64 * int(rng.integers(0, 4))
            span = st[i] * (dims[i] - 1) + span
        es = ELEM[dout := int(rng.integers(0, 3))]
        qo = rows(BASE, *st)
        ko = rows(BASE + es * st[1] * nq + (16 * int(rng.integers(-40, 40)) if rng.random() < 0.6 else 0), *st)
        want = meet(qo, nq, ko, nk, ext, es, es)
        assert cross(qo, nq, ko, nk, ext, dout) == want, (ext, nq, nk, st, dout, ko.data - BASE)
        seen.append(want)
    assert 200 < sum(seen) < 1900
