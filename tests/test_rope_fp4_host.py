"""Host checks of the rotary calls and of the 4-bit cache (no GPU: arguments
are refused before anything is launched; the fake device addresses below are
never dereferenced)."""

import ctypes as C
import os
import re

import numpy as np
import pytest

import rope_aware_quantized_gb300 as bg
from rope_aware_quantized_gb300 import _native

BASE, FAR = 1 << 20, 1 << 40
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def rope(cos=BASE, sin=BASE, n_pos=100, axes=1, axis=None, layout=0):
    d = _native.BgtqRope(cos, sin, n_pos, axes, None, layout)
    if axis is not None:
        d.keep = np.asarray(axis, np.uint8)
        d.axis = d.keep.ctypes.data
    return d


def rows(data=BASE, sb=1 << 16, sh=1 << 12, st=128):
    return _native.BgtqRows(data, sb, sh, st)


def fp4(groups=BASE, capacity=64, heads=2, page=0, n_pages=8, table=BASE, max_pages=None):
    d = _native.BgtqFp4Cache(groups, capacity, heads, None, 0, 0, 0)
    if page:
        d.page_table, d.max_pages, d.page_tokens, d.n_pages = table, max_pages or capacity // page, page, n_pages
    return d


def ref(x):
    return None if x is None else C.byref(x)


def outcome(rc):
    return rc, bg.lib().bgtq_last_error().decode()


def call_rows(r=None, pos=BASE, batch=1, t=4, q=None, qo=None, nq=2, k=None, ko=None, nk=0, din=0, dout=0, inverse=0):
    return outcome(bg.lib().bgtq_rope_rows(None, ref(r or rope()), pos, batch, t, ref(q or rows()), ref(qo or rows(FAR)), nq,
                                           ref(k), ref(ko), nk, din, dout, inverse, None))


def call_append(r=None, pos=BASE, k=None, v=None, batch=1, t=4, start=BASE, c=None, no_rope=False):
    return outcome(bg.lib().bgtq_fp4_append(None, None if no_rope else ref(r or rope()), pos, ref(k or rows()), ref(v or rows()),
                                            batch, t, start, ref(c or fp4()), None))


def call_attn(r=None, pos=BASE, q=None, group=4, batch=1, t=1, c=None, lens=BASE, max_len=64, out=BASE, dtype=1, scale=0.1,
              ws=BASE, ws_bytes=1 << 40, no_rope=False):
    return outcome(bg.lib().bgtq_fp4_attn(None, None if no_rope else ref(r or rope()), pos, ref(q or rows()), group, batch, t,
                                          ref(c or fp4()), lens, max_len, out, dtype, scale, ws, ws_bytes, None))


def plan(layout=0):
    return bg.bgtq_plan_create(np.full((2, 64), 3, np.uint8), np.ones((2, 64)), 4, 384, 3, 1, rope_layout=layout, host_only=True)


def call_rope_append(p, r=None, pos=BASE, k=None, v=None, batch=1, t=4, start=BASE):
    c = _native.BgtqCache(BASE, BASE, BASE, BASE, 64)
    return outcome(bg.lib().bgtq_rope_append(p.handle, None, ref(r or rope()), pos, ref(k or rows()), ref(v or rows()), batch, t,
                                             start, ref(c), None))


def test_every_declared_symbol_is_exported_and_bound():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "bgtq.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(bgtq_\w+)\s*\(", text))
    assert {"bgtq_rope_rows", "bgtq_fp4_attn", "bgtq_fp4_append"} <= names
    assert names == set(_native.EXPORTS)
    for n in names:
        assert hasattr(bg.lib(), n)


BAD_ROPE = [(dict(cos=None), "NULL"), (dict(sin=BASE + 4), "16-byte"), (dict(n_pos=0), "n_pos"), (dict(n_pos=1 << 31), "n_pos"),
            (dict(axes=0), "axes"), (dict(axes=5), "axes"), (dict(layout=2), "layout"),
            (dict(axes=2, axis=[0] * 63 + [2]), "axis of block 63")]


@pytest.mark.parametrize("bad,word", BAD_ROPE)
@pytest.mark.parametrize("call", [call_rows, call_append, call_attn, lambda r: call_rope_append(plan(), r)])
def test_rope_descriptor_refusals(call, bad, word):
    rc, msg = call(r=rope(**bad)) if call is not None else None
    assert rc == -1 and word in msg


BAD_ROWS = [(dict(data=None), "NULL"), (dict(data=BASE + 8), "16-byte"), (dict(st=132), "strides"), (dict(sh=4), "strides"),
            (dict(st=-128), "strides"), (dict(st=1 << 60), "range")]


@pytest.mark.parametrize("bad,word", BAD_ROWS)
def test_row_refusals(bad, word):
    for rc, msg in (call_rows(q=rows(**bad)), call_append(k=rows(**bad)), call_append(v=rows(**bad)),
                    call_attn(q=rows(**bad), t=2), call_rope_append(plan(), k=rows(**bad)), call_rope_append(plan(), v=rows(**bad)),
                    call_rows(k=rows(**bad), ko=rows(FAR), nk=2)):
        assert rc == -1 and word in msg


@pytest.mark.parametrize("kw,word", [
    (dict(pos=None), "pos is NULL"), (dict(batch=-1), ">= 0"), (dict(t=-1), ">= 0"), (dict(nq=-1), ">= 0"), (dict(din=3), "dtypes"),
    (dict(dout=-1), "dtypes"), (dict(inverse=2), "inverse"),
    (dict(qo=rows(FAR, st=0)), "overlap one another"), (dict(qo=rows(FAR, st=64)), "overlap one another"),
    (dict(qo=rows(FAR, sh=256, st=128)), "overlap one another"), (dict(qo=rows(FAR, sb=4096), batch=2), "overlap one another"),
    (dict(qo=rows(BASE + 256)), "q_out overlaps q"), (dict(qo=rows(BASE, st=256)), "q_out overlaps q"),
    (dict(qo=rows(), din=0, dout=2), "q_out overlaps q"),
    (dict(k=rows(), ko=rows(BASE + 16), nk=2), "k_out overlaps k"),
    (dict(k=rows(), nk=2), "k_out is NULL"),
])
def test_rope_rows_refusals(kw, word):
    rc, msg = call_rows(**kw)
    assert rc == -1 and word in msg


def test_calls_without_work():
    assert call_rows(batch=0)[0] == 0 and call_rows(t=0)[0] == 0 and call_rows(nq=0)[0] == 0
    assert call_append(batch=0)[0] == 0 and call_append(t=0)[0] == 0
    assert call_attn(batch=0)[0] == 0 and call_attn(t=0)[0] == 0
    assert call_rope_append(plan(), t=0)[0] == 0 and call_rope_append(plan(), batch=0)[0] == 0


def test_rope_append_refusals():
    assert call_rope_append(plan())[1].startswith("plan") or "host-only" in call_rope_append(plan())[1]
    rc, msg = call_rope_append(plan(layout=1))
    assert rc == -1 and "layout" in msg
    assert call_rope_append(plan(), batch=40000)[0] == -2
    assert "pos_start" in call_rope_append(plan(), start=None)[1]
    assert outcome(bg.lib().bgtq_rope_append(None, None, ref(rope()), BASE, ref(rows()), ref(rows()), 1, 1, BASE, None, None))[0] == -1


@pytest.mark.parametrize("bad,word", [
    (dict(groups=None), "NULL"), (dict(groups=BASE + 8), "16-byte"), (dict(capacity=24), "capacity"), (dict(capacity=0), "capacity"),
    (dict(capacity=(1 << 30) + 16), "capacity"), (dict(heads=0), "n_heads"), (dict(page=8), "page_tokens"),
    (dict(page=48, capacity=96), "page_tokens"), (dict(page=32, n_pages=0), "max_pages"), (dict(page=32, max_pages=3), "max_pages"),
    (dict(page=32, table=BASE + 2), "4-byte"),
])
def test_fp4_descriptor_refusals(bad, word):
    for rc, msg in (call_append(c=fp4(**bad)), call_attn(c=fp4(**bad)),
                    outcome(bg.lib().bgtq_fp4_dequant(None, ref(fp4(**bad)), 1, 0, 0, 0, 16, BASE, BASE))):
        assert rc == -1 and word in msg


@pytest.mark.parametrize("kw,code,word", [
    (dict(group=0), -1, "group"), (dict(group=9), -1, "group"), (dict(dtype=2), -1, "out_dtype"), (dict(scale=0.0), -1, "softmax_scale"),
    (dict(scale=float("nan")), -1, "softmax_scale"), (dict(scale=float("inf")), -1, "softmax_scale"), (dict(batch=-1), -1, ">= 0"),
    (dict(max_len=-1), -1, ">= 0"), (dict(lens=None), -1, "NULL"), (dict(out=None), -1, "NULL"), (dict(ws=None), -1, "NULL"),
    (dict(out=BASE + 8), -1, "out must"), (dict(ws=BASE + 128), -1, "256-byte"), (dict(ws_bytes=100), -4, "workspace"),
    (dict(batch=40000), -2, "65535"), (dict(no_rope=True), -1, "pos without rope"),
    (dict(t=1 << 28, q=rows(sh=1 << 40, st=128)), -2, "2^31"),
])
def test_fp4_attn_refusals(kw, code, word):
    rc, msg = call_attn(**kw)
    assert rc == code and word in msg


def test_fp4_append_refusals():
    assert call_append(no_rope=True)[0] == -1 and "pos without rope" in call_append(no_rope=True)[1]
    assert call_append(batch=65536)[0] == -2
    assert "pos_start" in call_append(start=None)[1]


def test_dequant_refusals():
    f = bg.lib().bgtq_fp4_dequant
    for args in ((1, 1, 0, 0, 16), (1, -1, 0, 0, 16), (1, 0, 2, 0, 16), (1, 0, 0, 8, 4), (1, 0, 0, 0, 80), (1, 0, 0, -1, 4)):
        assert f(None, ref(fp4()), *args, BASE, BASE) == -1
    assert f(None, ref(fp4()), 1, 0, 0, 5, 5, BASE, BASE) == 0


def test_table_refusals():
    f = np.ones(64)
    t = bg.lib().bgtq_rope_table
    assert t(None, None, 4, 1.0, BASE, BASE) == -1
    assert t(None, f.ctypes.data, 0, 1.0, BASE, BASE) == -1
    assert t(None, f.ctypes.data, 4, float("inf"), BASE, BASE) == -1
    assert t(None, f.ctypes.data, 4, 1.0, BASE + 4, BASE) == -1
    f[9] = np.nan
    assert t(None, f.ctypes.data, 4, 1.0, BASE, BASE) == -1 and "inv_freq[9]" in bg.lib().bgtq_last_error().decode()


def test_bytes():
    assert bg.bgtq_fp4_cache_bytes(2, 3, 64) == 2 * 3 * 4 * 2304
    assert bg.bgtq_fp4_cache_bytes(1, 0, 64) == 0
    for bad in ((0, 1, 64), (1, -1, 64), (1, 1, 24), (1, 1, -16)):
        with pytest.raises(bg.BgtqError):
            bg.bgtq_fp4_cache_bytes(*bad)
    for bad in ((0, 4, 1, 1, 64), (2, 9, 1, 1, 64), (2, 4, -1, 1, 64), (2, 4, 1, -1, 64), (2, 4, 1, 1, -1)):
        with pytest.raises(bg.BgtqError):
            bg.bgtq_fp4_attn_workspace(*bad)


def test_a_workspace_serves_smaller_calls():
    r = np.random.default_rng(0)
    for _ in range(300):
        H, G = int(r.integers(1, 9)), int(r.integers(1, 9))
        B, t, n = (int(2 ** r.uniform(0, m)) for m in (7, 12, 19))
        big = bg.bgtq_fp4_attn_workspace(H, G, B, t, n)
        b, s, m = int(r.integers(0, B + 1)), int(r.integers(0, t + 1)), int(r.integers(0, n + 1))
        assert bg.bgtq_fp4_attn_workspace(H, G, b, s, m) <= big
