"""GPU: the rotary operators at places that test_gpu_rope.py does not reach; bits are equal, as there."""

import numpy as np
import pytest

import rope_aware_quantized_gb300 as bg
from tests.test_gpu_rope import SECTIONS, i32, tables

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def seeded():
    torch.manual_seed(24)


@pytest.mark.parametrize("layout,axis", [(0, None), (1, SECTIONS)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_rows_into_other_heads_of_their_tensor(layout, axis, dtype):
    """Queries and keys of [B][T][heads][128] rotated into its other heads: the bits of a call with outputs apart, nothing else changed."""
    rope = bg.Rope(*tables(500), layout, axis)
    B, T, nq, nk = 2, 37, 6, 2
    pos = i32(np.random.default_rng(0).integers(0, 500, (rope.axes, B, T)))
    x = torch.randn((B, T, 2 * (nq + nk) + 1, 128), device="cuda").to(dtype)
    was = x.clone()
    part = lambda a, n: x[:, :, a:a + n].transpose(1, 2)  # noqa: E731
    q, k, qo, ko = part(0, nq), part(nq, nk), part(nq + nk, nq), part(2 * nq + nk, nk)
    want = [torch.empty((B, n, T, 128), dtype=dtype, device="cuda") for n in (nq, nk)]
    bg.bgtq_rope_rows(rope, pos, q, want[0], k, want[1])
    bg.bgtq_rope_rows(rope, pos, q, qo, k, ko)
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
    assert torch.equal(x[:, :, :nq + nk], was[:, :, :nq + nk]) and torch.equal(x[:, :, -1], was[:, :, -1])
    for bad in (dict(q_out=part(1, nq)), dict(k_out=qo[:, -nk:]), dict(k_out=part(nq + 1, nk))):
        with pytest.raises(bg.BgtqError, match="overlap"):
            bg.bgtq_rope_rows(**{**dict(rope=rope, pos=pos, q=q, q_out=qo, k=k, k_out=ko), **bad})
