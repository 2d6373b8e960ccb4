"""Host checks of the ragged serving step's entry points: every refusal is
made before any CUDA call (no GPU here, and no compute call is made)."""
import ctypes

import pytest
import torch

import kv_cache_mixed_kvq_b200 as kvq

BAD, UNSUP, OK = kvq.KVQ_ERR_INVALID_ARG, kvq.KVQ_ERR_UNSUPPORTED, kvq.KVQ_OK


def _desc(**kw):
    d = dict(batch=2, kv_heads=2, head_dim=128, capacity=64, bits_k=4, bits_v=2, group=64,
             flags=0, group_v=0, reserved=0, k_codes=0x1000, v_codes=0x2000, k_params=0x3000,
             v_params=0x4000, page_size=0, num_pages=0, block_table=None)
    d.update(kw)
    return kvq.KvqCacheDesc(*d.values())


PAGED = dict(flags=kvq.KVQ_FLAG_PAGED, page_size=32, num_pages=5, block_table=0x5000)


@pytest.mark.parametrize("batch,tokens,want", [
    (1, 0, 0), (1, 1, 1), (1, 16, 3), (1, 17, 3), (4, 3, 3), (64, 64, 64), (2, 1000, 66),
    (-1, 4, 0), (4, -1, 0), (2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1)])
def test_slot_map_entries(batch, tokens, want):
    assert kvq.kvq_slot_map_entries(batch, tokens) == want


@pytest.mark.parametrize("lens", [[(0, 1)], [(15, 17)], [(0, 0), (3, 40), (16, 32)],
                                  [(i, i + 2) for i in range(15, 80, 16)]])
def test_slot_map_entries_is_enough(lens):
    tiles = sum((n + 15) // 16 - o // 16 for o, n in lens if n > o)
    assert tiles <= kvq.kvq_slot_map_entries(len(lens), sum(n - o for o, n in lens))


def _plan(desc=None, **kw):
    a = dict(old=0x100, new=0x200, tokens=8, users=None, lens=0x300, cu=0x400, map=0x500,
             entries=8)
    a.update(kw)
    d = desc or _desc()
    return kvq.library().kvq_plan_append(
        ctypes.byref(d), a["old"], a["new"], a["tokens"], a["users"], a["lens"], a["cu"],
        a["map"], a["entries"], None)


def test_plan_refusals():
    for name in ("old", "new", "lens", "cu"):
        assert _plan(**{name: None}) == BAD
        assert _plan(**{name: 0x102}) == BAD
    assert _plan(tokens=-1) == BAD
    assert _plan(entries=3) == BAD               # fewer than kvq_slot_map_entries
    assert _plan(map=None) == BAD
    assert _plan(map=0x504) == BAD               # misaligned
    assert _plan(users=0x600) == BAD             # user counts without pages
    assert _plan(_desc(**PAGED)) == BAD          # pages without user counts
    assert _plan(_desc(**PAGED), users=0x602) == BAD
    assert _plan(lens=0x100) == BAD              # lens over old_lens, over new_lens
    assert _plan(lens=0x200) == BAD
    assert _plan(_desc(batch=8193)) == UNSUP
    assert _plan(_desc(capacity=2 ** 30 + 16)) == UNSUP
    assert _plan(_desc(head_dim=80)) == UNSUP
    assert _plan(_desc(reserved=1)) == BAD


def _append(desc=None, deq=False, **kw):
    a = dict(k=0x100, ks=256, v=0x200, vs=256, dt=1, tokens=8, map=0x500, entries=8)
    a.update(kw)
    d = desc or _desc()
    if deq:
        return kvq.library().kvq_dequantize_ragged(ctypes.byref(d), a["map"], a["entries"],
                                                   a["k"], a["v"], a["dt"], a["tokens"], None)
    return kvq.library().kvq_quantize_append_ragged(
        ctypes.byref(d), a["k"], a["ks"], a["v"], a["vs"], a["dt"], a["tokens"], a["map"],
        a["entries"], None)


@pytest.mark.parametrize("deq", [False, True])
def test_append_and_read_back_refusals(deq):
    for name in ("k", "v", "map"):
        assert _append(deq=deq, **{name: None}) == BAD
        assert _append(deq=deq, **{name: 0x108}) == BAD
    assert _append(deq=deq, dt=3) == BAD
    assert _append(deq=deq, tokens=-1) == BAD
    assert _append(deq=deq, entries=-1) == BAD
    assert _append(_desc(bits_k=3), deq=deq) == UNSUP
    # nothing to do: nothing is touched
    assert _append(deq=deq, tokens=0) == OK
    assert _append(deq=deq, entries=0) == OK


def test_append_strides():
    assert _append(ks=255) == BAD                # tokens overlap
    assert _append(vs=260) == BAD                # not 16 bytes apart
    assert _append(ks=258, dt=0) == BAD
    assert _append(ks=-256) == BAD


def _chunk(desc=None, **kw):
    a = dict(q=0x100, qs=1024, qt=1, hq=8, tokens=8, cu=0x200, lens=0x300, maxq=4, maxlen=64,
             causal=1, scale=0.0, out=0x400, ot=1, ws=None, wsb=0)
    a.update(kw)
    d = desc or _desc()
    return kvq.library().kvq_chunk_attention(
        ctypes.byref(d), a["q"], a["qs"], a["qt"], a["hq"], a["tokens"], a["cu"], a["lens"],
        a["maxq"], a["maxlen"], a["causal"], a["scale"], a["out"], a["ot"], a["ws"], a["wsb"],
        None)


def test_chunk_refusals():
    for name in ("q", "cu", "lens", "out"):
        assert _chunk(**{name: None}) == BAD
    assert _chunk(q=0x108) == BAD
    assert _chunk(out=0x108) == BAD
    assert _chunk(cu=0x202) == BAD
    assert _chunk(lens=0x302) == BAD
    assert _chunk(qt=4) == BAD
    assert _chunk(ot=-1) == BAD
    assert _chunk(hq=7) == BAD                   # not a multiple of Hkv
    assert _chunk(hq=0) == BAD
    assert _chunk(qs=1016) == BAD                # tokens overlap
    assert _chunk(qs=1028) == BAD                # not 16 bytes apart
    assert _chunk(tokens=-1) == BAD
    assert _chunk(maxq=-1) == BAD
    assert _chunk(maxlen=-1) == BAD
    assert _chunk(scale=float("nan")) == BAD
    assert _chunk(_desc(capacity=24)) == BAD
    assert _chunk(tokens=2 ** 28) == UNSUP       # rows past 32 bits
    assert _chunk(_desc(batch=16385)) == UNSUP
    assert _chunk(_desc(capacity=2 ** 30 + 16), maxlen=2 ** 30 + 16) == UNSUP
    # (query tile, key tile) pairs past 32 bits
    assert _chunk(_desc(capacity=2 ** 26), tokens=2 ** 25, maxlen=2 ** 26) == UNSUP
    assert _chunk(tokens=0, q=None) == OK


def test_python_calls_want_cuda_tensors():
    z = torch.zeros
    cache = kvq.KVCache(2, 2, 128, 64, 4, 2, 64, *(z(16, dtype=torch.uint8) for _ in range(4)))
    i2, i3 = z(2, dtype=torch.int32), z(3, dtype=torch.int32)
    slots, x = z((4, 4), dtype=torch.int32), z((4, 2, 128))
    for call in (lambda: kvq.kvq_plan_append(cache, i2, i2, 4),
                 lambda: kvq.kvq_quantize_append_ragged(cache, x, x, slots),
                 lambda: kvq.kvq_dequantize_ragged(cache, slots, 4),
                 lambda: kvq.kvq_chunk_attention(cache, x, i3, i2, 4, 64)):
        with pytest.raises(ValueError):
            call()


def test_pools_of_many_pages():
    """The number of pages is not bound by a grid's limits (batch rows are)."""
    page = kvq.kvq_cache_bytes(1, 2, 128, 32, 4, 2, 64, kvq.KVQ_K_CODES)
    assert kvq.kvq_cache_bytes(200000, 2, 128, 32, 4, 2, 64, kvq.KVQ_K_CODES) == 200000 * page
    lib = kvq.library()
    assert lib.kvq_validate_cache(ctypes.byref(_desc(**dict(PAGED, num_pages=200000)))) == OK
    assert lib.kvq_validate_cache(ctypes.byref(_desc(batch=65536))) == UNSUP


def test_caches_copy_without_their_descriptor():
    """The descriptor kept by a cache follows its fields and stays out of copies."""
    import copy
    cache = kvq.KVCache(2, 2, 128, 64, 4, 2, 64, *(torch.zeros(16, dtype=torch.uint8)
                                                   for _ in range(4)))
    cache.__dict__["_desc"] = ((0,) * 5, kvq.KvqCacheDesc())
    other = copy.deepcopy(cache)
    assert "_desc" not in other.__dict__ and other.batch == 2
    assert other.k_codes.data_ptr() != cache.k_codes.data_ptr()
    cache.rotate_keys = True
    assert "_desc" not in cache.__dict__
