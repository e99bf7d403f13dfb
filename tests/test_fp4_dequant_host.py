"""Host check of the 4-bit cache's inspection (no GPU): a cache on another device than the current one is refused."""

import types

import pytest

import rope_aware_quantized_gb300 as bg

torch = pytest.importorskip("torch")


class Groups:
    """A stand-in for a cache's tensor on cuda:1."""
    is_cuda, device = True, "cuda:1"

    def get_device(self):
        return 1


def test_a_cache_on_another_device_is_refused(monkeypatch):
    calls = []
    monkeypatch.setattr(bg, "_device", lambda x: 0)
    monkeypatch.setattr(bg, "lib", lambda: types.SimpleNamespace(bgtq_fp4_dequant=lambda *a: calls.append(a) or 0))
    cache = types.SimpleNamespace(groups=Groups(), batch=1, desc=bg._native.BgtqFp4Cache())
    for stream in (None, 0, 5):
        with pytest.raises(ValueError, match="current device is cuda:0"):
            bg.bgtq_fp4_dequant(cache, 0, 0, 0, 16, stream=stream)
    assert not calls
    cache.groups = torch.zeros(1, dtype=torch.uint8)  # (a cache of the host)
    with pytest.raises(ValueError):
        bg.bgtq_fp4_dequant(cache, 0, 0, 0, 16, stream=5)
