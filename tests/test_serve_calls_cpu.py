"""Host checks of the serving step's binding and build (no GPU here)."""
import pytest
import torch

import kv_cache_mixed_kvq_b200 as kvq
from kv_cache_mixed_kvq_b200 import build


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


def test_tensors_of_another_device_are_refused(monkeypatch):
    """The kernels would read and write its addresses on the cache's device."""
    cache = _cache(monkeypatch)
    monkeypatch.setattr(kvq, "_on_current", lambda device: None)
    monkeypatch.setattr(kvq, "_stream_ptr", lambda stream: None)
    q, cu, lens = torch.zeros(4, 4, 128), torch.zeros(3, dtype=torch.int32), \
        torch.zeros(2, dtype=torch.int32)

    def attend(**kw):
        # (bounds of no token and length: nothing is launched)
        return kvq.kvq_chunk_attention(cache, kw.get("q", q)[:0], kw.get("cu", cu),
                                       kw.get("lens", lens), 0, 0, out=kw.get("out", q)[:0],
                                       workspace=kw.get("workspace", torch.zeros(64)))

    attend()
    for name, t in (("q", q), ("cu", cu), ("lens", lens), ("out", q),
                    ("workspace", torch.zeros(64))):
        with pytest.raises(ValueError):
            attend(**{name: t.to("meta")})
    cache.v_codes = cache.v_codes.to("meta")
    with pytest.raises(ValueError):
        attend()


def _report(kernel, registers):
    return (f"ptxas info    : Compiling entry function '{kernel}' for 'sm_100a'\n"
            f"ptxas info    : Function properties for {kernel}\n"
            "    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads\n"
            f"ptxas info    : Used {registers} registers, used 1 barriers\n")


def test_build_checks_the_registers_of_the_split_kernels():
    """A compiler that gives the kernel fewer registers is noticed by the build;
    one that stays within the same allocation is no reason to refuse."""
    good = "_ZN3kvq5chunk12chunk_kernelINS0_3CfgE"
    for n in (65, 70, 72):
        build.check_launch_registers(_report("combine_kernel", 32) + _report(good, n))
    for n in (32, 64, 73, 80):
        with pytest.raises(RuntimeError, match=f"{n} registers"):
            build.check_launch_registers(_report(good, 72) + _report(good, n))
    with pytest.raises(RuntimeError, match="no report"):
        build.check_launch_registers(_report("combine_kernel", 72))
