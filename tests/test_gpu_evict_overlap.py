"""GPU: an eviction refuses written buffers that meet each other, or records
that meet what it reads, before it launches anything."""

import pytest

import rope_aware_quantized_gb300 as bg

from tests.test_gpu_bounded import bare_layer, lens32

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

H, B, CAP, KEEP = 2, 2, 64, 32


@pytest.mark.parametrize("first,second", [
    ("kept", "dst_scores"), ("kept", "dst_lens"), ("dst_scores", "dst_lens"), ("kept", "k_codes"), ("kept", "v_norm"),
    ("dst_scores", "v_codes"), ("dst_lens", "k_norm"), ("k_codes", "v_codes"), ("v_norm", "k_norm"),
    ("v_codes", "scores"), ("k_norm", "seq_lens"), ("k_codes", "source v_codes"),
])
def test_written_buffers_that_meet(first, second):
    plan = bare_layer(H, 384, 3).plan
    src, dst = bg.Cache(plan, B, CAP), bg.Cache(plan, B, KEEP)
    bufs = dict(scores=torch.rand((B, H, CAP), device="cuda"), seq_lens=lens32([CAP, 40]),
                dst_scores=torch.zeros((B, H, KEEP), device="cuda"), dst_lens=lens32([-7, -7]),
                kept=torch.full((B, H, KEEP), -9, dtype=torch.int32, device="cuda"))

    def call():
        bg.bgtq_evict(plan, src, bufs["scores"], bufs["seq_lens"], CAP, KEEP, 2, 5, dst, bufs["dst_scores"], bufs["dst_lens"],
                      bufs["kept"])

    def get(name):
        return getattr(src, name[7:]) if name.startswith("source ") else getattr(dst, name) if name in vars(dst) else bufs[name]

    # the smaller of the two becomes a part of the larger's memory
    a, b = get(first), get(second)
    small, large = (first, b) if a.nbytes <= b.nbytes else (second, a)
    assert not small.startswith("source ")
    old = get(small)
    over = large.view(-1).view(torch.uint8)[:old.nbytes].view(old.dtype).view(old.shape)
    if small in vars(dst):
        setattr(dst, small, over)
        setattr(dst.desc, small, over.data_ptr())
    else:
        bufs[small] = over
    watched = [x.clone() for x in (dst.k_codes, dst.v_codes, dst.k_norm, dst.v_norm, *bufs.values())]
    with pytest.raises(bg.BgtqError, match="overlaps"):
        call()
    torch.cuda.synchronize()
    for x, y in zip(watched, (dst.k_codes, dst.v_codes, dst.k_norm, dst.v_norm, *bufs.values())):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
