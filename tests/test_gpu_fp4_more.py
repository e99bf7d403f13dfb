"""GPU: the 4-bit cache at places that test_gpu_fp4.py does not reach; its helpers, and its tolerances."""

import types

import numpy as np
import pytest

import rope_aware_quantized_gb300 as bg
from oracle import rope_fp4_oracle as F
from tests.test_gpu_fp4 import Case, gen, group_rows, i32, status

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def seeded():
    torch.manual_seed(23)


def check(c, out, half, units):
    """Checks those (sequence, query head)s of a case, each as a case of its own."""
    for b, a in units:
        one = Case.__new__(Case)
        one.H, one.G, one.t, one.lens, n = 1, 1, c.t, [c.lens[b]], -(-c.lens[b] // 16)
        rows = torch.from_numpy(group_rows(c.cache, b, a // c.G)[:n]).cuda()
        one.cache = types.SimpleNamespace(groups=c.cache.groups.view(-1, F.GROUP_BYTES)[rows].flatten(), capacity=16 * n, page_tokens=0, n_kv_heads=1)
        one.q = c.q[b:b + 1, a:a + 1]
        one.check(out[b:b + 1, a:a + 1], half)


def filled(B, H, G, t, lens, cap, page, seed, n_pages=0, spread=1.0):
    """A Case whose sequences are appended in one call of max(lens) positions a sequence."""
    c = Case.__new__(Case)
    c.H, c.G, c.t, c.lens, c.seq = H, G, t, [int(n) for n in lens], i32(lens)
    c.cache = bg.Fp4Cache(H, B, cap, page_tokens=page, n_pages=n_pages)
    top = max(c.lens)
    if n_pages:  # only the pages that are needed
        each = -(-top // page)
        c.cache.page_table.fill_(-1)
        c.cache.page_table[:, :each] = torch.randperm(n_pages, generator=gen(seed), device="cuda")[:B * each].view(B, each).to(torch.int32)
    k, v = (torch.randn((B, H, top, 128), generator=gen(seed + i), device="cuda").half() for i in (1, 2))
    bg.bgtq_fp4_append(k, v, i32(np.zeros(B)), c.cache)
    c.q = torch.randn((B, H * G, t, 128), generator=gen(seed + 3), device="cuda").half() * spread
    return c


@pytest.mark.parametrize("t", [1, 3, 5])
def test_many_rows_under_a_large_virtual_length(t):
    """2048 (sequence, head)s in a paged cache of 2^20 virtual positions a sequence: 8, 24 and 40 rows a head."""
    rng = np.random.default_rng(t)
    lens = rng.integers(t, 301, 256)
    lens[0] = 300
    c = filled(256, 8, 8, t, lens, 1 << 20, 256, t, n_pages=600)
    st = status()
    out = c.run(True, max_len=1 << 20, status=st)
    check(c, out, True, {(int(b), int(a)) for b, a in zip(rng.integers(0, 256, 25), rng.integers(0, 64, 25))})
    assert st.item() == 0


# (sequences, KV heads, bound): where the tiles are split unevenly, the parts of a head in tiles
UNEVEN = [(10, 8, 8192, (43, 21)), (15, 4, 16384, (52, 52, 24))]


@pytest.mark.parametrize("B,H,top,parts", UNEVEN)
@pytest.mark.parametrize("t,half", [(20, True), (20, False), (33, True), (40, False)])  # 80, 132 and 160 rows
def test_uneven_parts_of_a_head(B, H, top, parts, t, half):
    """Heads whose tiles are cut into equal parts and a smaller one, with lengths that end before, at and behind each border."""
    assert sum(parts) == top // 128
    ends = [128 * sum(parts[:i + 1]) for i in range(len(parts) - 1)]
    rng = np.random.default_rng(top + t)
    lens = [top, top - 1] + [e + d for e in ends for d in (-1, 0, 1, t, 200)] + [1, t]
    lens = (lens + rng.integers(1, top, B).tolist())[:B]
    c = filled(B, H, 4, t, lens, top, 0, seed=t)
    out = c.run(half, max_len=top)
    check(c, out, half, {(b, (5 * b + 1) % (4 * H)) for b in range(B)} | {(0, 0), (0, 4 * H - 1)})
    assert torch.equal(out, c.run(half, max_len=top))


@pytest.mark.parametrize("t", [1, 5, 40])  # 8, 40 and 320 rows a head
@pytest.mark.parametrize("page", [16, 32])
@pytest.mark.parametrize("half", [False, True])
def test_an_unmapped_page_is_reported_and_touches_no_other_sequence(t, page, half):
    c = Case(2, 8, t, [320, 500], 512, page, seed=page + t)
    st = status()
    good = c.run(half, status=st)
    assert st.item() == 0
    for entry in (-1, c.cache.n_pages, 1 << 30):
        c.cache.page_table[0, 1] = entry
        out = c.run(half, status=st.zero_())
        assert st.item() == bg.STATUS_PAGE_RANGE
        assert torch.equal(out[1], good[1])
    # pages behind the last position are not looked at
    c.cache.page_table[1, -(-500 // page):] = -1
    c.lens, c.seq = [16, 500], i32([16, 500])
    out = c.run(half, status=st.zero_())
    assert st.item() == 0 and torch.equal(out[1], good[1])


@pytest.mark.parametrize("t", [5, 40])  # 40 and 320 rows a head, whose tiles are split and joined
@pytest.mark.parametrize("half", [False, True])
def test_a_captured_call_with_parts_replayed(t, half):
    """Lengths, queries and positions changed on the device between replays, eager calls with the same workspace between them."""
    top = 6000
    c = filled(3, 2, 8, t, [top, 1, 2000], 6016, 64, seed=t)
    rope = bg.Rope(*bg.bgtq_rope_table(1e6 ** (-np.arange(64) / 64), 7000))
    pos = torch.zeros((3, t), dtype=torch.int32, device="cuda")
    ws = torch.zeros(bg.bgtq_fp4_attn_workspace(2, 8, 3, t, top), dtype=torch.uint8, device="cuda")
    dtype = torch.float16 if half else torch.float32
    out, two = (torch.empty((3, 16, t, 128), dtype=dtype, device="cuda") for _ in range(2))
    st = status()

    def call(o, **kw):
        bg.bgtq_fp4_attn(c.q, c.cache, c.seq, top, o, ws, rope=rope, pos=pos, status=st, **kw)

    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        call(out)
        call(two, softmax_scale=0.01)
    rng = np.random.default_rng(t)
    for i in range(12):
        lens = rng.integers(0, top + 1, 3)
        lens[i % 3] = (0, 1, top, t, 128, 129)[i % 6]
        c.seq.copy_(i32(lens))
        pos.copy_(i32(rng.integers(0, 7000, (3, t))))
        c.q.normal_()
        graph.replay()
        want, want2 = torch.empty_like(out), torch.empty_like(out)
        call(want)
        call(want2, softmax_scale=0.01)
        assert torch.equal(out, want) and torch.equal(two, want2)
        c.lens = lens.tolist()
        if i % 4 == 2:
            turned = torch.empty_like(c.q)
            bg.bgtq_rope_rows(rope, pos, c.q, turned)
            c.q.copy_(turned)
            check(c, out, half, {(b, 5 * b + i % 5) for b in range(3) if lens[b]})
    assert st.item() == 0


@pytest.mark.parametrize("t", [1, 3, 20])
def test_sequences_that_share_pages(t):
    """Two sequences over the same pages of a prefix, and their own from there: the outputs of sequences with copies."""
    c = Case(2, 4, t, [700, 700, 700], 704, 64, seed=t)
    apart = c.cache.groups.clone()
    P, table = c.cache.page_tokens // 16, c.cache.page_table
    g = c.cache.groups.view(-1, 2 * P * F.GROUP_BYTES)  # a pool page a row
    for i in range(8):
        g[table[1, i].long()] = g[table[0, i].long()]
    want = c.run(False)
    c.cache.groups.copy_(apart)
    table[1, :8] = table[0, :8]
    assert torch.equal(c.run(False), want)
