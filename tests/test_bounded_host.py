"""Host checks of the bounded-cache calls (no GPU: arguments are checked
before the plan, and the fake device addresses below are never
dereferenced)."""

import ctypes
import functools

import numpy as np
import pytest

import rope_aware_quantized_gb300 as bg

BASE = 1 << 20
OUT = 1 << 24
FAR = 1 << 40  # other buffers
H, G = 2, 4


@functools.lru_cache(maxsize=None)  # (kept: a plan's handle lives as long as its object)
def plan(bpk=384, bv=3):
    return bg.bgtq_plan_create(np.full((H, 64), bpk // 128, np.uint8), np.ones((H, 64)), G, bpk, bv, 1, host_only=True)


def desc(base=BASE, capacity=128, recent=0, page=0, n_pages=8, table=BASE):
    d = bg._native.BgtqCache(base, base + (1 << 28), base + (2 << 28), base + (3 << 28), capacity)
    if recent:
        d.k_recent, d.recent = base, recent
    if page:
        d.page_table, d.max_pages, d.page_tokens, d.n_pages = table, capacity // page, page, n_pages
    return d


def err():
    return bg.lib().bgtq_last_error().decode()


def window(p=None, q=BASE, kn=None, vn=None, pos=None, batch=1, max_len=100, sinks=4, win=32, out=OUT, out_dtype=1,
           scale=0.1, ws=BASE, ws_bytes=1 << 30, lens=BASE, **kw):
    d = desc(**kw)
    rc = bg.lib().bgtq_decode_window_attn((p or plan()).handle, None, q, kn, vn, pos, ctypes.byref(d), lens, max_len, batch,
                                          sinks, win, out, out_dtype, scale, ws, ws_bytes, None)
    return rc, err()


def score(p=None, q=BASE, kn=None, vn=None, pos=None, batch=1, max_len=100, sin=BASE, sout=BASE, out=OUT, out_dtype=1,
          scale=0.1, ws=BASE, ws_bytes=1 << 30, lens=BASE, **kw):
    d = desc(**kw)
    rc = bg.lib().bgtq_decode_score_attn((p or plan()).handle, None, q, kn, vn, pos, ctypes.byref(d), lens, max_len, batch,
                                         sin, sout, out, out_dtype, scale, ws, ws_bytes, None)
    return rc, err()


@pytest.mark.parametrize("call", [window, score])
def test_decode_valid_arguments_reach_the_plan_check(call):
    rc, msg = call()
    assert rc == -1 and "host-only" in msg
    rc, msg = call(kn=BASE, vn=BASE, pos=BASE)
    assert rc == -1 and "host-only" in msg
    assert call(batch=0)[0] == 0


@pytest.mark.parametrize("call", [window, score])
@pytest.mark.parametrize("kw,code,frag", [
    (dict(max_len=-1), -1, ">= 0"),
    (dict(batch=-1), -1, ">= 0"),
    (dict(batch=65536), -2, "65535"),
    (dict(q=None), -1, "NULL"),
    (dict(lens=None), -1, "NULL"),
    (dict(out=None), -1, "NULL"),
    (dict(ws=None), -1, "NULL"),
    (dict(kn=BASE), -1, "together"),
    (dict(kn=BASE, vn=BASE), -1, "together"),
    (dict(kn=BASE + 2, vn=BASE, pos=BASE), -1, "8-byte"),
    (dict(q=BASE + 2), -1, "q must be"),
    (dict(ws=BASE + 8), -1, "workspace"),
    (dict(out=OUT + 2), -1, "out must be"),
    (dict(out_dtype=2), -1, "out_dtype"),
    (dict(scale=0.0), -1, "softmax_scale"),
    (dict(scale=float("nan")), -1, "softmax_scale"),
    (dict(capacity=127), -1, "even"),
    (dict(recent=200), -1, "recent"),
])
def test_decode_bad_arguments_are_rejected(call, kw, code, frag):
    rc, msg = call(**kw)
    assert rc == code and frag in msg, (rc, msg)


@pytest.mark.parametrize("call", [window, score])
def test_decode_widths_that_have_no_instance(call):
    assert call(p=plan(512))[0] == -2
    assert call(p=plan(384, 5))[0] == -2


@pytest.mark.parametrize("kw,frag", [(dict(sinks=-1), "sinks"), (dict(win=0), "window"), (dict(win=-5), "window")])
def test_window_bad_masks(kw, frag):
    rc, msg = window(**kw)
    assert rc == -1 and frag in msg


@pytest.mark.parametrize("kw,frag", [
    (dict(sin=None), "NULL"), (dict(sout=None), "NULL"),
    (dict(sin=BASE + 4), "8-byte"), (dict(sout=BASE + 4), "8-byte"),
    (dict(sin=BASE, sout=BASE + 8), "overlap"),                            # one array shifted against the other
    (dict(sin=BASE + H * 128 * 4 - 8, sout=BASE), "overlap"),
])
def test_score_bad_score_arrays(kw, frag):
    rc, msg = score(**kw)
    assert rc == -1 and frag in msg
    rc, msg = score(sin=BASE, sout=BASE + H * 128 * 4)
    assert "host-only" in msg


def test_workspace_sizes():
    p, n = plan(), ctypes.c_size_t()
    L = bg.lib()
    assert L.bgtq_decode_window_workspace(p.handle, 1, 1 << 20, 4, 100, ctypes.byref(n)) == 0
    small = n.value
    assert L.bgtq_decode_window_workspace(p.handle, 1, 1 << 20, 4, 1 << 20, ctypes.byref(n)) == 0
    assert 0 < small <= n.value == bg.bgtq_decode_attn_workspace(p, 1, 1 << 20)
    assert bg.bgtq_decode_score_workspace(p, 2, 1000) >= bg.bgtq_decode_attn_workspace(p, 2, 1000) + 2 * H * G * (1008 * 4 + 8)
    for bad in ((-1, 10, 0, 1), (1, -1, 0, 1), (1, 10, -1, 1), (1, 10, 0, 0)):
        assert L.bgtq_decode_window_workspace(p.handle, *bad, ctypes.byref(n)) == -1
    assert L.bgtq_decode_score_workspace(p.handle, 1, -1, ctypes.byref(n)) == -1
    for bad in ((-1, 10, 0), (1, -1, 0), (1, 10, -1), (1, 10, 11)):
        assert L.bgtq_prefill_score_workspace(p.handle, *bad, ctypes.byref(n)) == -1


def prefill(q=BASE, k=BASE, v=BASE, batch=1, t=100, sinks=4, win=32, out=OUT, out_dtype=0, scale=0.1, lse=None, **kw):
    d = desc(**kw)
    rc = bg.lib().bgtq_prefill_window_attn(plan().handle, None, q, k, v, batch, t, sinks, win, ctypes.byref(d), out, out_dtype,
                                           scale, lse, None)
    return rc, err()


def pscore(q=BASE, k=BASE, lse=BASE, batch=1, t=100, row0=0, sinks=4, win=32, scale=0.1, scores=OUT, stride=128, ws=BASE,
           ws_bytes=1 << 30):
    rc = bg.lib().bgtq_prefill_score(plan().handle, None, q, k, lse, batch, t, row0, sinks, win, scale, scores, stride, ws,
                                     ws_bytes, None)
    return rc, err()


def test_prompt_calls_valid_arguments_and_no_ops():
    for call in (prefill, pscore):
        rc, msg = call()
        assert rc == -1 and "host-only" in msg
        assert call(t=0)[0] == 0 and call(batch=0)[0] == 0


@pytest.mark.parametrize("kw,code,frag", [
    (dict(t=200), -3, "capacity"), (dict(t=-1), -1, ">= 0"), (dict(q=BASE + 8), -1, "16-byte"), (dict(out=OUT + 8), -1, "16-byte"),
    (dict(lse=BASE + 2), -1, "lse"), (dict(out_dtype=2), -1, "out_dtype"), (dict(scale=-1.0), -1, "softmax_scale"),
    (dict(win=0), -1, "window"), (dict(sinks=-1), -1, "sinks"), (dict(batch=70000), -2, "65535"),
    (dict(batch=65535, t=5000, capacity=1 << 20), -2, "2^31"), (dict(v=None), -1, "NULL"),
])
def test_prefill_bad_arguments(kw, code, frag):
    rc, msg = prefill(**kw)
    assert rc == code and frag in msg, (rc, msg)


@pytest.mark.parametrize("kw,code,frag", [
    (dict(t=-1), -1, ">= 0"), (dict(row0=-1), -1, "row0"), (dict(row0=101), -1, "row0"), (dict(q=BASE + 8), -1, "16-byte"),
    (dict(k=BASE + 8), -1, "16-byte"), (dict(lse=None), -1, "NULL"), (dict(scores=None), -1, "NULL"),
    (dict(scores=OUT + 2), -1, "4-byte"), (dict(stride=99), -1, "stride"), (dict(scale=float("inf")), -1, "softmax_scale"),
    (dict(win=0), -1, "window"), (dict(sinks=-1), -1, "sinks"), (dict(batch=40000), -2, "65535"),
    (dict(batch=30000, t=10000, stride=10000), -2, "2^31"), (dict(t=8388481, stride=8388481), -2, "8388480"),
    (dict(t=4096, stride=4096, ws_bytes=0), -4, "workspace"), (dict(t=4096, stride=4096, ws=None), -1, "workspace"),
])
def test_prefill_score_bad_arguments(kw, code, frag):
    rc, msg = pscore(**kw)
    assert rc == code and frag in msg, (rc, msg)


def evict(scores=BASE, lens=BASE, max_len=128, batch=1, keep=32, sinks=4, recent=8, dst_scores=FAR, dst_lens=FAR, kept=FAR,
          src=None, dst=None):
    s, d = src or desc(), dst or desc(FAR, 64)
    rc = bg.lib().bgtq_evict(plan().handle, None, ctypes.byref(s), scores, lens, max_len, batch, keep, sinks, recent,
                             ctypes.byref(d), dst_scores, dst_lens, kept, None)
    return rc, err()


def test_evict_valid_arguments():
    assert "host-only" in evict()[1]
    assert "host-only" in evict(keep=12)[1]
    assert "host-only" in evict(keep=1000, max_len=50)[1]  # a budget past the destination, but no sequence is longer
    assert evict(batch=0)[0] == 0
    # one pool, two page tables
    assert "host-only" in evict(src=desc(page=16, table=BASE), dst=desc(capacity=64, page=16, table=BASE + 64))[1]


@pytest.mark.parametrize("kw,code,frag", [
    (dict(keep=0), -1, "keep"), (dict(keep=1 << 31), -1, "keep"), (dict(sinks=-1), -1, "sinks"), (dict(recent=-1), -1, "recent"),
    (dict(sinks=30, recent=3), -1, "at most keep"), (dict(max_len=-1), -1, ">= 0"), (dict(batch=70000), -2, "65535"),
    (dict(scores=None), -1, "NULL"), (dict(kept=None), -1, "NULL"), (dict(dst_lens=None), -1, "NULL"),
    (dict(scores=BASE + 2), -1, "4-byte"), (dict(keep=65), -3, "destination"),
    (dict(dst_scores=BASE), -1, "overlaps"), (dict(dst_lens=BASE), -1, "overlaps"),
    (dict(dst=desc(BASE, 64)), -1, "overlap"), (dict(dst=desc(BASE + 16, 64)), -1, "overlap"),
    (dict(src=desc(recent=8)), -2, "recent-key"), (dict(dst=desc(FAR, 64, recent=8)), -2, "recent-key"),
    (dict(src=desc(page=16), dst=desc(capacity=64, page=16)), -1, "overlap"),        # one page table
    (dict(src=desc(page=16), dst=desc(capacity=64)), -1, "overlap"),                 # a pool and a contiguous cache in it
])
def test_evict_bad_arguments(kw, code, frag):
    rc, msg = evict(**kw)
    assert rc == code and frag in msg, (rc, msg)


def test_binding_checks_tensors():
    import torch
    p = plan()
    q = torch.zeros(1, H * G, 128, dtype=torch.float16)
    with pytest.raises(ValueError, match="shape"):
        bg.bgtq_decode_window_attn(p, q[:, :3], None, None, 10, 0, 4, q, q)
    with pytest.raises(ValueError, match="CUDA"):
        bg.bgtq_decode_window_attn(p, q, None, None, 10, 0, 4, q, q)
    with pytest.raises(ValueError, match="contiguous"):
        bg.bgtq_prefill_score(p, q.view(1, H * G, 1, 128).expand(1, H * G, 4, 128), q, q, q)


@pytest.mark.parametrize("batch", [1, 3, 13, 37])
def test_a_workspace_serves_every_shorter_length(batch):
    p = plan()
    for size in (lambda n: bg.bgtq_decode_window_workspace(p, batch, n, 20, 5000),
                 lambda n: bg.bgtq_decode_window_workspace(p, batch, 1 << 20, 20, n),
                 lambda n: bg.bgtq_decode_window_workspace(p, batch, n, 0, 1 << 40),
                 lambda n: bg.bgtq_decode_score_workspace(p, batch, n)):
        last = 0
        for n in [*range(1, 20000, 61), *range(20000, 700000, 4001)]:
            assert size(n) >= last, n
            last = size(n)
    most, far = 2 ** 31 - 1, 2 ** 63 - 1  # (no sequence is longer)
    assert bg.bgtq_decode_window_workspace(p, batch, far, far, far) == bg.bgtq_decode_window_workspace(p, batch, most, far, far)
    assert bg.bgtq_decode_score_workspace(p, batch, far) == bg.bgtq_decode_score_workspace(p, batch, most)


def test_prompt_scores_refuse_scales_whose_log_sum_exp_does_not_fit():
    rc, msg = pscore(scale=9e-7)
    assert rc == -2 and "1e-6" in msg
    rc, msg = pscore(scale=1e-6)
    assert rc == -1 and "host-only" in msg
