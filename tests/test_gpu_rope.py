"""GPU: rotary tables, rows and the rotated append.

Tolerances.  The tables are functions of 64-bit angles rounded once: half a
step of float32, 2^-24 of the value, plus 2^-40 for the functions themselves.
Rotated rows are float32 operations in a fixed order, one rounding each, so
they equal the same operations in numpy bit for bit; against float64 an
element is off by three half steps of float32 of its two products (3 2^-24
(|lo| + |hi|), cos and sin at most 1) and half a step of the output type.
Records, norms and recent keys are equal, bit for bit.
"""

import numpy as np
import pytest

import rope_aware_quantized_gb300 as bg
from oracle import rope_fp4_oracle as F
from rope_aware_quantized_gb300 import synth

from tests.test_gpu_parity import dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

INV = 1e6 ** (-np.arange(64) / 64)
SECTIONS = [0] * 16 + [1] * 24 + [2] * 24
MIXED = [i % 3 for i in range(64)]
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
HALF_STEP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}


@pytest.fixture(autouse=True)
def seeded():
    torch.manual_seed(21)


def tables(n, inv=INV):
    return bg.bgtq_rope_table(inv, n)


def positions(rng, axes, B, T, n_pos):
    return rng.integers(0, n_pos, (axes, B, T)).astype(np.int32)


def i32(x):
    return torch.as_tensor(np.asarray(x, np.int32)).cuda()


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("n,scale", [(1, 1.0), (5, 0.5), (4097, 1.2)])
def test_table(n, scale):
    cos, sin = bg.bgtq_rope_table(INV, n, scale)
    a = np.arange(n)[:, None] * INV[None]
    for got, want in ((cos, scale * np.cos(a)), (sin, scale * np.sin(a))):
        assert (np.abs(got.cpu().numpy() - want) <= 2.0 ** -24 * np.abs(want) + 2.0 ** -40).all()


def test_table_far_positions():
    n = (1 << 21) + 3
    cos, _ = bg.bgtq_rope_table(INV, n)
    a = np.arange(n - 500, n)[:, None] * INV[None]  # angles of 2 million radians keep 64-bit accuracy
    want = np.cos(a)
    assert (np.abs(cos[n - 500:].cpu().numpy() - want) <= 2.0 ** -24 * np.abs(want) + 2.0 ** -29).all()


def expected(x, cos, sin, pos, layout, axis, inverse, out):
    """numpy, float32, one rounding an operation; x [B][h][T][128] float32 values, pos [axes][B][T]."""
    y = F.rope(x, cos, sin, pos[:, :, None, :].repeat(x.shape[1], 2), layout, axis, inverse)
    return torch.from_numpy(y).to(DTYPES[out])


@pytest.mark.parametrize("B,nq,nk,T,axis,layout,din,dout,inverse", [
    (1, 4, 1, 1, None, 0, "f16", "f16", False),
    (3, 1, 0, 1, None, 1, "f16", "f16", False),
    (2, 16, 2, 33, None, 0, "f16", "f16", True),
    (2, 7, 1, 65, SECTIONS, 0, "f16", "f16", False),
    (1, 5, 3, 130, MIXED, 1, "bf16", "f16", False),
    (1, 8, 8, 31, MIXED, 0, "f32", "f32", True),
    (2, 3, 2, 64, None, 1, "f32", "bf16", False),
    (1, 2, 1, 17, SECTIONS, 1, "bf16", "bf16", False),
    (1, 2, 1, 17, None, 0, "bf16", "f32", False),
    (1, 2, 2, 9, None, 0, "f16", "f32", False),
    (1, 2, 2, 9, None, 0, "f16", "bf16", True),
    (1, 2, 2, 9, None, 0, "f32", "f16", True),
    (1, 40, 8, 2500, None, 0, "f16", "f16", False),
])
def test_rows(B, nq, nk, T, axis, layout, din, dout, inverse):
    rng = np.random.default_rng(B * 1000 + T)
    cos, sin = tables(700)
    pos = positions(rng, 1 if axis is None else 3, B, T, 700)
    # a projection's output: [B][T][heads][128], queries, keys and something else side by side
    x = torch.randn((B, T, nq + nk + 1, 128), device="cuda").to(DTYPES[din])
    q, k = x[:, :, :nq].transpose(1, 2), x[:, :, nq:nq + nk].transpose(1, 2)
    qo = torch.full((B, nq, T, 128), 7.0, dtype=DTYPES[dout], device="cuda")
    ko = torch.full((B, nk, T, 128), 7.0, dtype=DTYPES[dout], device="cuda")
    st = status()
    rope = bg.Rope(cos, sin, layout, axis)
    bg.bgtq_rope_rows(rope, i32(pos), q, qo, k if nk else None, ko if nk else None, inverse, status=st)
    c, s = cos.cpu().numpy(), sin.cpu().numpy()
    for got, src in ((qo, q), (ko, k)):
        xs = src.float().cpu().numpy()
        assert torch.equal(got.cpu(), expected(xs, c, s, pos, layout, axis, inverse, dout))
        exact = F.rope(xs, c, s, pos[:, :, None, :].repeat(xs.shape[1], 2), layout, axis, inverse, exact=True)
        lo, hi = (xs[..., :64], xs[..., 64:]) if layout == 0 else (xs[..., 0::2], xs[..., 1::2])
        mag = np.abs(lo) + np.abs(hi)
        mag = np.concatenate([mag, mag], -1) if layout == 0 else np.repeat(mag, 2, -1)
        tol = (3 * 2.0 ** -24 + HALF_STEP[dout] * (1 + 2.0 ** -20)) * mag + 2.0 ** -25
        assert (np.abs(got.float().cpu().numpy() - exact) <= tol).all()
    assert st.item() == 0


def test_rows_in_place_and_back():
    cos, sin = tables(300)
    rope = bg.Rope(cos, sin)
    pos = i32(np.random.default_rng(0).integers(0, 300, (2, 50)))
    x = torch.randn((2, 50, 6, 128), device="cuda")
    q, k = x[:, :, :4].transpose(1, 2), x[:, :, 4:].transpose(1, 2)
    was = x.clone()
    want = torch.empty((2, 4, 50, 128), device="cuda")
    bg.bgtq_rope_rows(rope, pos, q, want)
    bg.bgtq_rope_rows(rope, pos, q, q, k, k)
    assert torch.equal(q, want)
    bg.bgtq_rope_rows(rope, pos, q, q, k, k, inverse=True)
    # two rotations of three half steps each, of |lo| + |hi|, on top of cos^2 + sin^2 = 1 +- 2^-23
    assert ((x - was).abs() <= 16 * 2.0 ** -24 * was.abs().max()).all()


def test_inverse_is_the_gradient():
    """<J g, d> = <g, rotate(d)> for the inverse of g as J^T g, and against central differences."""
    cos, sin = tables(100)
    rope = bg.Rope(cos, sin, 1, MIXED)
    pos = i32(positions(np.random.default_rng(1), 3, 1, 8, 100))
    x, g, d = (torch.randn((1, 2, 8, 128), device="cuda") for _ in range(3))

    def turn(v, inverse=False):
        out = torch.empty_like(v)
        bg.bgtq_rope_rows(rope, pos, v, out, inverse=inverse)
        return out.double()

    grad = turn(g, True)
    n = 2048
    tol = 8 * 2.0 ** -24 * (g.double().abs() * 2 * d.double().abs()).sum().item() + n * 2.0 ** -24
    assert abs((grad * d.double()).sum() - (g.double() * turn(d)).sum()) <= tol
    h = 0.5  # the map is linear: a difference of any width is exact but for roundings
    diff = (g.double() * (turn(x + h * d) - turn(x - h * d))).sum() / (2 * h)
    tol = 8 * 2.0 ** -24 * (g.double().abs() * 2 * (x.double().abs() + d.double().abs())).sum().item() / h
    assert abs((grad * d.double()).sum() - diff) <= tol


def test_rows_outside_the_tables_are_left():
    cos, sin = tables(64)
    q = torch.randn((1, 3, 6, 128), device="cuda").half()
    out = torch.full_like(q, 9.0)
    pos = np.array([[[0, 63, 64, -1, 5, 2**31 - 1]], [[1, 2, 3, 4, 64, 0]]], np.int32)
    st = status()
    bg.bgtq_rope_rows(bg.Rope(cos, sin, 0, [0] * 32 + [1] * 32), i32(pos), q, out, status=st)
    assert st.item() == bg.STATUS_ROPE_RANGE
    got = out.cpu()
    assert (got[:, :, 2:] == 9).all()
    want = expected(q[:, :, :2].float().cpu().numpy(), cos.cpu().numpy(), sin.cpu().numpy(), pos[:, :, :2], 0, [0] * 32 + [1] * 32, False, "f16")
    assert torch.equal(got[:, :, :2], want)


def test_broadcast_input_and_padded_output():
    cos, sin = tables(64)
    row = torch.randn((1, 1, 1, 128), device="cuda").half()
    q = row.expand(2, 3, 5, 128)  # strides 0
    big = torch.full((2, 5, 4, 192), 3.0, device="cuda").half()
    out = big[:, :, 1:4, 32:160].transpose(1, 2)
    pos = np.arange(10, dtype=np.int32).reshape(1, 2, 5)
    bg.bgtq_rope_rows(bg.Rope(cos, sin), i32(pos), q, out)
    want = expected(q.float().cpu().numpy(), cos.cpu().numpy(), sin.cpu().numpy(), pos, 0, None, False, "f16")
    assert torch.equal(out.cpu(), want)
    assert (big[:, :, 0] == 3).all() and (big[..., :32] == 3).all() and (big[..., 160:] == 3).all()


def test_python_refusals():
    cos, sin = tables(64)
    rope, pos = bg.Rope(cos, sin), i32(np.zeros((1, 4)))
    q = torch.zeros((1, 2, 4, 128), dtype=torch.float16, device="cuda")
    ok = torch.empty_like(q)
    for bad in (dict(q=q[..., :64]), dict(q=q.cpu()), dict(q_out=ok[:, :1]), dict(q=q.to(torch.float64)), dict(pos=pos[:, :3]),
                dict(pos=pos.long()), dict(pos=None), dict(k=q), dict(k=q.float(), k_out=ok), dict(q=q[..., ::2].expand(1, 2, 4, 64)),
                dict(rope=None), dict(status=torch.zeros(1, device="cuda", dtype=torch.int64))):
        a = dict(rope=rope, pos=pos, q=q, q_out=ok)
        a.update(bad)
        with pytest.raises((ValueError, bg.BgtqError)):
            bg.bgtq_rope_rows(**a)
    for bad in (dict(axis=[0] * 63), dict(axis=[0] * 63 + [4]), dict(sections=(16, 16)), dict(axis=[0] * 64, sections=(64,))):
        with pytest.raises(ValueError):
            bg.Rope(cos, sin, **bad)
    with pytest.raises(ValueError):
        bg.Rope(cos.cpu(), sin.cpu())
    with pytest.raises(ValueError):
        bg.Rope(cos, sin[:3])
    with pytest.raises(ValueError):
        bg.bgtq_rope_table(INV[:3], 4)
    assert bg.Rope(cos, sin, sections=(16, 24, 24)).axis.tolist() == SECTIONS


# ----------------------------------------------------------------- the rotated append


def layer(seed, H, bpk, bv, layout):
    li = synth.layer_inputs(seed, 0, H, 1, 8, 1e5, 1.0, n_calib=128, rope_layout=layout)
    be = [bg.bgtq_alloc_bits(li.calib[h], bpk, rope_layout=layout) for h in range(H)]
    return bg.bgtq_plan_create(np.stack([b for b, _ in be]), np.stack([e for _, e in be]), 2, bpk, bv, 5 + seed, rope_layout=layout)


def filled(plan, B, cap, page, recent, seed):
    """A cache whose buffers hold random bytes, and a copy of it."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    c = bg.Cache(plan, B, cap, page_tokens=page, recent=recent)
    for name in ("k_codes", "v_codes"):
        getattr(c, name).copy_(torch.randint(0, 256, getattr(c, name).shape, generator=g, device="cuda", dtype=torch.uint8))
    if page:
        c.page_table.copy_(torch.randperm(c.n_pages, generator=g, device="cuda").to(torch.int32).view_as(c.page_table))
    d = bg.Cache(plan, B, cap, page_tokens=page, recent=recent)
    for x in (c, d):
        out.append(x)
    same(c, d, copy=True)
    return out


NAMES = ("k_codes", "v_codes", "k_norm", "v_norm", "k_recent")


def same(c, d, copy=False):
    for n in NAMES:
        if copy:
            getattr(d, n).copy_(getattr(c, n))
        else:
            assert torch.equal(getattr(c, n), getattr(d, n)), n
    if c.page_table is not None:
        d.page_table.copy_(c.page_table)


@pytest.mark.parametrize("B,H,T,bpk,bv,cap,page,starts,axis,layout,recent", [
    (1, 1, 1, 384, 3, 64, 0, [0], None, 0, 0),
    (3, 2, 1, 256, 2, 64, 16, [0, 17, 63], None, 0, 0),
    (2, 2, 1, 384, 3, 64, 0, [5, 8], None, 1, 8),
    (2, 3, 5, 256, 4, 128, 32, [3, 100], SECTIONS, 0, 4),
    (1, 2, 63, 128, 3, 256, 0, [9], MIXED, 1, 0),
    (2, 2, 64, 384, 3, 256, 0, [0, 7], None, 0, 16),
    (2, 1, 65, 256, 2, 256, 64, [1, 30], None, 1, 10),
    (1, 2, 1000, 384, 1, 2048, 16, [33], SECTIONS, 0, 0),
    (1, 2, 1000, 128, 2, 2048, 0, [32], MIXED, 0, 1000),
    (1, 1, 300, 256, 4, 512, 0, [0], MIXED, 1, 0),
    (1, 2, 40, 512, 5, 64, 0, [3], None, 0, 0),  # widths that only the small append takes
    (1, 2, 100, 512, 5, 128, 0, [3], None, 1, 0),
])
def test_append_equals_the_two_calls(B, H, T, bpk, bv, cap, page, starts, axis, layout, recent):
    rng = np.random.default_rng(T)
    plan = layer(T, H, bpk, bv, layout)
    cos, sin = tables(3000)
    rope = bg.Rope(cos, sin, layout, axis)
    pos = i32(positions(rng, rope.axes, B, T, 3000))
    x = torch.randn((B, T, 2 * H + 1, 128), device="cuda").half() * 3
    k, v = x[:, :, 1:H + 1].transpose(1, 2), x[:, :, H + 1:].transpose(1, 2)
    a, b = filled(plan, B, cap, page, recent, T)
    st, start = status(), i32(starts)
    bg.bgtq_rope_append(plan, rope, pos, k, v, start, a, status=st)
    kr = torch.empty((B, H, T, 128), dtype=torch.float16, device="cuda")
    bg.bgtq_rope_rows(rope, pos, k, kr)
    bg.bgtq_quantize_append(plan, kr, v.contiguous(), start, b)
    same(a, b)
    assert st.item() == 0
    if axis is None:  # positions left out: the cache's own
        own = start[:, None] + torch.arange(T, dtype=torch.int32, device="cuda")
        bg.bgtq_rope_append(plan, rope, own.contiguous(), k, v, start, b)
        bg.bgtq_rope_append(plan, rope, None, k, v, start, a)
        same(a, b)


@pytest.mark.parametrize("T", [4, 130])
def test_append_skips_tokens_outside_the_tables(T):
    """A token with a position outside the tables keeps its slot's old record; its V pair's other half is merged."""
    plan = layer(3, 2, 384, 3, 0)
    cos, sin = tables(50)
    rope = bg.Rope(cos, sin)
    p = np.arange(T) % 50
    bad = [1, 2, T - 1]
    p[bad] = [50, -1, 1 << 30]
    k, v = (torch.randn((1, 2, T, 128), device="cuda").half() for _ in range(2))
    a, b = filled(plan, 1, 256, 0, 0, 1)
    st = status()
    bg.bgtq_rope_append(plan, rope, i32(p[None]), k, v, i32([3]), a, status=st)
    assert st.item() == bg.STATUS_ROPE_RANGE
    for t in range(T):  # one at a time, without those
        if t not in bad:
            bg.bgtq_rope_append(plan, rope, i32(p[None, t:t + 1]), k[:, :, t:t + 1], v[:, :, t:t + 1], i32([3 + t]), b)
    same(a, b)


def test_append_past_the_capacity_and_unmapped_pages():
    plan = layer(4, 1, 256, 2, 0)
    rope = bg.Rope(*tables(100))
    k, v = (torch.randn((2, 1, 70, 128), device="cuda").half() for _ in range(2))
    a, b = filled(plan, 2, 128, 16, 0, 2)
    a.page_table[1, 2] = -1
    b.page_table.copy_(a.page_table)
    st = status()
    bg.bgtq_rope_append(plan, rope, None, k, v, i32([100, 0]), a, status=st)
    assert st.item() == bg.STATUS_APPEND_CAPACITY | bg.STATUS_PAGE_RANGE
    kr = torch.empty_like(k)
    bg.bgtq_rope_rows(rope, i32(np.tile(np.arange(70), (2, 1))), k, kr)
    bg.bgtq_quantize_append(plan, kr, v, i32([100, 0]), b)
    same(a, b)


def test_a_run_on_the_packed_cache():
    """A prompt rotated and prefilled, the cache cut, then steps whose rotary positions run on
    while the slots start again behind the cut: the records and outputs of steps on keys and
    queries rotated beforehand."""
    H, G, T, keep = 2, 2, 200, 64
    plan = layer(9, H, 384, 3, 0)
    rope = bg.Rope(*tables(400))
    x = torch.randn((1, T, H * G + 2 * H, 128), device="cuda").half()
    q, k, v = (x[:, :, a:b].transpose(1, 2) for a, b in ((0, H * G), (H * G, H * G + H), (H * G + H, H * G + 2 * H)))
    pos = torch.arange(T, dtype=torch.int32, device="cuda").view(1, T)
    qr, kr = torch.empty(q.shape, dtype=q.dtype, device="cuda"), torch.empty(k.shape, dtype=k.dtype, device="cuda")
    bg.bgtq_rope_rows(rope, pos, q, qr, k, kr)
    full, out = bg.Cache(plan, 1, T), torch.empty_like(qr)
    lse = torch.empty((1, H * G, T), device="cuda")
    bg.bgtq_prefill_window_attn(plan, qr, kr, v.contiguous(), full, 0, T, out, lse=lse)
    other = bg.Cache(plan, 1, T)
    bg.bgtq_rope_append(plan, rope, pos, k, v, i32([0]), other)
    same(full, other)
    scores = torch.empty((1, H, T), device="cuda")
    bg.bgtq_prefill_score(plan, qr, kr, lse, scores, torch.zeros(max(16, bg.bgtq_prefill_score_workspace(plan, 1, T)), dtype=torch.uint8, device="cuda"))
    caches = []
    for _ in range(2):
        c = bg.Cache(plan, 1, 128)
        lens = i32([0])
        bg.bgtq_evict(plan, full, scores, i32([T]), T, keep, 2, 10, c, torch.zeros((1, H, 128), device="cuda"), lens,
                      torch.empty((1, H, keep), dtype=torch.int32, device="cuda"))
        assert lens.item() == keep
        caches.append(c)
    a, b = caches
    ws = [torch.zeros(bg.bgtq_decode_attn_workspace(plan, 1, 128), dtype=torch.uint8, device="cuda") for _ in range(2)]
    oa, ob = (torch.empty((1, H * G, 128), device="cuda") for _ in range(2))
    for i in range(5):
        q, k, v = (torch.randn((1, n, 1, 128), device="cuda").half() for n in (H * G, H, H))
        pos, slot, n = i32([[T + i]]), i32([keep + i]), i32([keep + i + 1])
        qr, kr = torch.empty_like(q), torch.empty_like(k)
        bg.bgtq_rope_rows(rope, pos, q, qr)
        bg.bgtq_rope_append(plan, rope, pos, k, v, slot, a)
        bg.bgtq_decode_attn(plan, qr.squeeze(2), a, n, 128, oa, ws[0])
        c, s = rope.cos.cpu().numpy(), rope.sin.cpu().numpy()
        kr = expected(k.float().cpu().numpy(), c, s, np.array([[[T + i]]]), 0, None, False, "f16").cuda()
        qn = expected(q.float().cpu().numpy(), c, s, np.array([[[T + i]]]), 0, None, False, "f16").cuda()
        bg.bgtq_decode_step(plan, qn.squeeze(2), kr.squeeze(2), v.squeeze(2), slot, b, n, 128, ob, ws[1])
        assert torch.equal(oa, ob)
        same(a, b)


def test_rotation_captured_replayed_and_on_another_stream():
    plan = layer(6, 2, 384, 3, 0)
    rope = bg.Rope(*tables(200))
    pos = i32(np.arange(12).reshape(2, 6))
    k, v, q = (torch.randn((2, n, 6, 128), device="cuda").half() for n in (2, 2, 4))
    qo, start = torch.empty_like(q), i32([0, 9])
    a, b = filled(plan, 2, 64, 0, 0, 3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        bg.bgtq_rope_rows(rope, pos, q, qo)
        bg.bgtq_rope_append(plan, rope, pos, k, v, start, a)
    for rep in range(3):
        k.normal_()
        q.normal_()
        pos.add_(rep)
        torch.cuda.synchronize()
        graph.replay()
        want = torch.empty_like(q)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            bg.bgtq_rope_rows(rope, pos, q, want)
            bg.bgtq_rope_append(plan, rope, pos, k, v, start, b)
        torch.cuda.synchronize()
        assert torch.equal(qo, want)
        same(a, b)


def test_rows_past_2_to_the_31_elements():
    cos, sin = tables(64)
    B, T, n = 1, 1 << 18, 65  # 2.18e9 elements
    q = torch.zeros((B, T, n, 128), dtype=torch.float16, device="cuda")
    q[:, -3:] = torch.randn((B, 3, n, 128), device="cuda").half()
    pos = torch.zeros((B, T), dtype=torch.int32, device="cuda")
    pos[:, -3:] = i32([[5, 6, 63]])
    v = q.transpose(1, 2)
    tail = v[:, :, -3:].float().cpu().numpy()
    bg.bgtq_rope_rows(bg.Rope(cos, sin), pos, v, v)
    want = expected(tail, cos.cpu().numpy(), sin.cpu().numpy(), np.array([[[5, 6, 63]]]), 0, None, False, "f16")
    assert torch.equal(v[:, :, -3:].cpu(), want)
