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


def sampled(c, half, rng, some, **kw):
    """Runs a case and checks `some` of its (sequence, query head)s, each as a case of its own."""
    out = c.run(half, **kw)
    B, hq = c.q.shape[:2]
    for b, a in {(int(b), int(a)) for b, a in zip(rng.integers(0, B, some), rng.integers(0, hq, some))}:
        one = Case.__new__(Case)
        one.H, one.G, one.t, one.lens, n = 1, 1, c.t, [c.lens[b]], -(-c.lens[b] // 16)
        rows = torch.from_numpy(group_rows(c.cache, b, a // c.G)[:n]).cuda()
        one.cache = types.SimpleNamespace(groups=c.cache.groups.view(-1, F.GROUP_BYTES)[rows].flatten(), capacity=16 * n, page_tokens=0, n_kv_heads=1)
        one.q = c.q[b:b + 1, a:a + 1]
        one.check(out[b:b + 1, a:a + 1], half)
    return out


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
    sampled(c, True, rng, 25, max_len=1 << 20, status=st)
    assert st.item() == 0
