"""Host checks of the serving step's binding and build (no GPU here)."""
import pytest
import torch

import kv_cache_mixed_kvq_b200 as kvq


def _cache(monkeypatch):
    """A cache of host tensors that the binding takes for device ones."""
    def pointer(t, name):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return t.data_ptr()

    monkeypatch.setattr(kvq, "_dev_ptr", pointer)
    return kvq.KVCache(2, 2, 128, 64, 4, 2, 64, *(torch.zeros(16, 16, dtype=torch.uint8)
                                                  for _ in range(4)))


def test_a_descriptor_is_the_callers_own(monkeypatch):
    """One that is edited (for a view of some rows, say) leaves the cache's
    later calls as they were."""
    cache = _cache(monkeypatch)
    d = cache.desc()
    d.batch, d.k_codes = 1, d.k_codes + 16
    again = cache.desc()
    assert again.batch == 2 and again.k_codes == cache.k_codes.data_ptr()
    assert cache._kept_desc() is cache._kept_desc()  # (the calls share one)


def test_buffers_are_checked_again_when_their_layout_changes(monkeypatch):
    cache = _cache(monkeypatch)
    cache.desc()
    cache.v_params.t_()  # the same address
    with pytest.raises(ValueError):
        cache.desc()
    cache.v_params.t_()
    cache.desc()
