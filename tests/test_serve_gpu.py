"""GPU parity of the ragged serving step: page planning and slot maps against
a plain loop; ragged append bit for bit against kvq_quantize_append (itself
bit-identical to the oracle) and against the oracle's read-back; chunk
attention against 64-bit attention over the cached values; the three of them
run together over steps that grow, verify, roll back and finish rows; calls
captured into a CUDA graph."""
import random

import numpy as np
import pytest
import torch

import kv_cache_mixed_kvq_b200 as kvq
from kv_cache_mixed_kvq_b200 import workloads
from tests.serve_util import (DT, assert_close, attention_reference, fill, i32, make_cache,
                              plan_reference, random_tables, tokens)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ planning
def _check_plan(old, new, table, users, P, cap, total=None):
    """One planning call against the plain loop; returns the error flags."""
    B = len(old)
    cache = kvq.KVCache.allocate(B, 1, 64, cap, 2, 2, 64, page_size=P, num_pages=len(users),
                                 block_table=torch.from_numpy(table.copy()))
    u = torch.from_numpy(users.copy()).cuda()
    ref = plan_reference(old, new, table.tolist(), users.tolist(), P, cap, B)
    total = ref[1][-1] if total is None else total
    lens, cu, m = kvq.kvq_plan_append(cache, i32(old), i32(new), total, u)
    flags = kvq.kvq_device_error_flags()
    assert lens.tolist() == ref[0]
    assert cu.tolist() == ref[1]
    assert cache.block_table.tolist() == ref[3]
    assert u.tolist() == ref[4]
    got = m.tolist()
    assert got[:len(ref[2])] == ref[2]
    assert all(e == [0, 0, 0, 0] for e in got[len(ref[2]):])
    return flags, ref[5]


@pytest.mark.parametrize("B,P,cap,hi,grow,spare", [
    (1, 32, 32, 0, 1, 1), (1, 32, 4096, 4000, 96, 4), (3, 64, 256, 200, 56, 9),
    (64, 64, 2048, 1900, 1, 70), (257, 32, 1024, 900, 100, 900), (1000, 32, 2048, 1990, 58, 3000),
    (1025, 128, 1024, 800, 200, 2100), (5, 256, 65536, 65000, 400, 12000),
    (3000, 32, 512, 400, 100, 9000), (8192, 32, 64, 40, 20, 9000)])
def test_plan_matches_plain_loop(B, P, cap, hi, grow, spare):
    rng = np.random.default_rng(B + P)
    old = rng.integers(0, hi + 1, B).tolist()
    new = [int(min(cap, o + rng.integers(0, grow + 1))) if rng.random() < 0.7
           else int(rng.integers(0, o + 1)) for o in old]
    table, users = random_tables(rng, old, P, cap, spare)
    flags, refused = _check_plan(old, new, table, users, P, cap)
    assert flags == 0 and not refused


@pytest.mark.parametrize("B,spare", [(4, 2), (300, 100), (2000, 700)])
def test_plan_without_enough_pages(B, spare):
    rng = np.random.default_rng(spare)
    old = rng.integers(0, 500, B).tolist()
    new = [int(o + rng.integers(0, 90)) for o in old]
    table, users = random_tables(rng, old, 32, 1024, spare)
    flags, refused = _check_plan(old, new, table, users, 32, 1024)
    assert flags == kvq.KVQ_DEVERR_NO_PAGE and refused


def test_plan_shared_pages():
    # rows 0 and 1 share a whole page, rows 2 and 3 a partly filled one
    table = np.array([[5, 1, -1, -1], [5, 2, -1, -1], [3, -1, -1, -1], [3, -1, -1, -1]], np.int32)
    users = np.array([0, 1, 1, 2, 0, 2, 0, 0], np.int32)
    flags, refused = _check_plan([40, 64, 20, 20], [70, 65, 21, 20], table, users, 32, 128)
    assert flags == kvq.KVQ_DEVERR_NO_PAGE and refused == {2}
    # the other user leaves in the same step: the page is this row's alone
    flags, refused = _check_plan([40, 64, 20, 20], [0, 0, 40, 0], table, users, 32, 128)
    assert flags == 0 and not refused


def test_plan_invalid_lengths():
    table, users = random_tables(np.random.default_rng(0), [10, 10, 10], 32, 64, 3)
    for bad, flag in ((-1, kvq.KVQ_DEVERR_BAD_POS), (65, kvq.KVQ_DEVERR_SEQ_LEN)):
        flags, refused = _check_plan([10, 10, 10], [40, bad, 33], table, users, 32, 64)
        assert flags == flag and refused == {1}


def test_plan_pages_outside_the_pool():
    table, users = random_tables(np.random.default_rng(0), [10, 40], 32, 64, 3)
    table[0, 0] = 99
    cache = kvq.KVCache.allocate(2, 1, 64, 64, 2, 2, 64, page_size=32, num_pages=len(users),
                                 block_table=torch.from_numpy(table))
    u = torch.from_numpy(users).cuda()
    lens, cu, m = kvq.kvq_plan_append(cache, i32([10, 40]), i32([12, 41]), 3, u)
    assert kvq.kvq_device_error_flags() == kvq.KVQ_DEVERR_BAD_PAGE
    assert lens.tolist() == [10, 41] and m.tolist()[0][2:] == [2, 1]
    # returned: counted once, the entry cleared
    lens, _, _ = kvq.kvq_plan_append(cache, i32([10, 41]), i32([0, 41]), 0, u)
    assert kvq.kvq_device_error_flags() == kvq.KVQ_DEVERR_BAD_PAGE
    assert cache.block_table[0, 0].item() == -1 and u.tolist() == users.tolist()


def test_plan_more_tokens_than_announced():
    table, users = random_tables(np.random.default_rng(1), [0, 0], 32, 64, 4)
    cache = kvq.KVCache.allocate(2, 1, 64, 64, 2, 2, 64, page_size=32, num_pages=len(users),
                                 block_table=torch.from_numpy(table))
    _, _, m = kvq.kvq_plan_append(cache, i32([0, 0]), i32([3, 20]), 5,
                                  torch.from_numpy(users).cuda())
    assert kvq.kvq_device_error_flags() == kvq.KVQ_DEVERR_CAPACITY
    assert [e[2:] for e in m.tolist()][:2] == [[0, 3], [3, 2]]
    assert all(e[3] == 0 or e[2] + e[3] <= 5 for e in m.tolist())


def test_plan_slot_layout():
    cache = kvq.KVCache.allocate(3, 1, 64, 128, 2, 2, 64)
    lens, cu, m = kvq.kvq_plan_append(cache, i32([0, 30, 9]), i32([17, 30, 0]), 17)
    assert lens.tolist() == [17, 30, 0] and cu.tolist() == [0, 17, 17, 17]
    assert m.tolist() == [[0, 0, 0, 16], [0, 16, 16, 1]] + [[0, 0, 0, 0]] * (m.shape[0] - 2)


# ------------------------------------------------------- append and read-back
SHAPES = [  # D, bk, bv, G, Gv, rotate, dtype, P
    (128, 4, 2, 64, 0, False, "bf16", 64), (128, 8, 4, 32, 128, True, "f32", 0),
    (128, 2, 8, 128, 0, False, "f16", 32), (64, 4, 4, 32, 64, False, "bf16", 128),
    (64, 2, 2, 64, 0, True, "f16", 32), (64, 8, 8, 32, 0, False, "f32", 0),
    (128, 4, 2, 32, 64, True, "bf16", 32), (128, 8, 2, 128, 0, False, "f32", 256)]


def _appended_pair(shape, old, new, seed, wide=False):
    """Two caches with the same bytes: one appended with the ragged call, one
    row by row with kvq_quantize_append through a one-row table."""
    D, bk, bv, G, gv, rot, dt, P = shape
    B, Hkv, cap = len(old), 3, 1024
    want = [max(o, n) for o, n in zip(old, new)]
    cache, users = make_cache(B, Hkv, D, cap, bk, bv, G, gv, rot, P, 5, want=want)
    for t in (cache.k_codes, cache.v_codes, cache.k_params, cache.v_params):
        t.copy_(torch.randint(0, 256, t.shape, dtype=torch.uint8))  # bytes to be kept
    kvq.kvq_plan_append(cache, i32([0] * B), i32(old), sum(old), users)
    total = sum(n - o for o, n in zip(old, new))
    _, cu, slots = kvq.kvq_plan_append(cache, i32(old), i32(new), total, users)
    bufs = [t.clone() for t in (cache.k_codes, cache.v_codes, cache.k_params, cache.v_params)]
    if wide:  # slices of one projection's output
        x = tokens(total, 3 * Hkv, D, dt, seed, 2.0, 3.0)
        k, v = x[:, Hkv:2 * Hkv], x[:, 2 * Hkv:]
        assert total < 2 or not k.is_contiguous()
    else:
        k = tokens(total, Hkv, D, dt, seed, 2.0, 3.0)
        v = tokens(total, Hkv, D, dt, seed + 1)
    kvq.kvq_quantize_append_ragged(cache, k, v, slots)
    at = 0
    for b, (o, n) in enumerate(zip(old, new)):
        if n == o:
            continue
        if P:
            one = kvq.KVCache(1, Hkv, D, cap, bk, bv, G, *bufs, rotate_keys=rot, group_v=gv,
                              page_size=P, num_pages=cache.num_pages,
                              block_table=cache.block_table[b:b + 1].contiguous())
        else:
            cut = [t.view(B, -1)[b] for t in bufs]
            one = kvq.KVCache(1, Hkv, D, cap, bk, bv, G, *cut, rotate_keys=rot, group_v=gv)
        kvq.kvq_quantize_append(one, k[at:at + n - o].transpose(0, 1).unsqueeze(0).contiguous(),
                                v[at:at + n - o].transpose(0, 1).unsqueeze(0).contiguous(),
                                i32([o]))
        at += n - o
    assert kvq.kvq_device_error_flags() == 0
    return cache, bufs, slots, total


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("old,new", [
    ([0], [1]), ([5, 0, 31, 100], [6, 1, 32, 101]), ([0, 7, 300, 16], [257, 7, 401, 48]),
    ([15, 33, 1], [17, 160, 16])])
def test_append_ragged_bits(shape, old, new):
    cache, bufs, _, _ = _appended_pair(shape, old, new, seed=len(old))
    for name, t in zip(("k_codes", "v_codes", "k_params", "v_params"), bufs):
        assert torch.equal(getattr(cache, name), t), name


def test_append_ragged_strided_inputs():
    cache, bufs, _, _ = _appended_pair(SHAPES[0], [3, 60], [90, 61], seed=3, wide=True)
    for name, t in zip(("k_codes", "v_codes", "k_params", "v_params"), bufs):
        assert torch.equal(getattr(cache, name), t), name


def test_append_ragged_degenerate_groups():
    """Constant groups, zeros of both signs, and the largest values."""
    cache, _ = make_cache(1, 1, 128, 64, 4, 2, 32)
    ref = kvq.KVCache.allocate(1, 1, 128, 64, 4, 2, 32)
    k = torch.zeros(4, 1, 128)
    k[0] = -0.0
    k[1] = 7.25
    k[2, 0, ::2] = 65504.0
    k[2, 0, 1::2] = -65504.0
    k[3, 0, 0] = 1e-30
    v = -k
    _, _, slots = kvq.kvq_plan_append(cache, i32([0]), i32([4]), 4)
    kvq.kvq_quantize_append_ragged(cache, k.cuda(), v.cuda(), slots)
    kvq.kvq_quantize_append(ref, k.view(1, 1, 4, 128).cuda(), v.view(1, 1, 4, 128).cuda(), i32([0]))
    assert torch.equal(cache.k_codes, ref.k_codes) and torch.equal(cache.k_params, ref.k_params)
    assert torch.equal(cache.v_codes, ref.v_codes) and torch.equal(cache.v_params, ref.v_params)


@pytest.mark.parametrize("D,bk,bv,G,gv,rot", [
    (128, 4, 2, 64, 0, False), (128, 8, 4, 32, 128, False), (64, 2, 8, 32, 0, False),
    (128, 2, 4, 64, 0, True), (64, 8, 2, 64, 0, True)])
def test_dequantize_matches_oracle(ora, D, bk, bv, G, gv, rot):
    Hkv, cap, T = 2, 64, 37
    cache, _ = make_cache(1, Hkv, D, cap, bk, bv, G, gv, rot)
    hc = ora.HostCache(1, Hkv, D, cap, bk, bv, G, rotate_keys=rot, group_v=gv or None)
    k, v = tokens(T, Hkv, D, "bf16", 1, 2.0, 3.0), tokens(T, Hkv, D, "bf16", 2)
    kb, dt = workloads.as_bits(k.transpose(0, 1).unsqueeze(0).contiguous().cpu())
    vb, _ = workloads.as_bits(v.transpose(0, 1).unsqueeze(0).contiguous().cpu())
    hc.quantize_append(kb, vb, [0], dtype=dt)
    _, _, slots = kvq.kvq_plan_append(cache, i32([0]), i32([T]), T)
    kvq.kvq_quantize_append_ragged(cache, k, v, slots)
    for name, out in (("f32", torch.float32), ("bf16", torch.bfloat16), ("f16", torch.float16)):
        kd, vd = kvq.kvq_dequantize_ragged(cache, slots, T, out)
        half = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[name]
        for h in range(Hkv):
            rk = np.asarray(hc.dequant_slot(0, 0, h, T), np.float64)
            rv = np.asarray(hc.dequant_slot(1, 0, h, T), np.float64)
            # one binary32 rounding of code * scale + zero, one to the output
            # type; unrotating sums D stored values in log2(D) rounded steps
            tol_v = (2.0 ** -24 + half) * np.abs(rv) + 2.0 ** -25
            tol_k = (2.0 ** -24 + half) * np.abs(rk) + 2.0 ** -25
            if rot:
                mag = np.abs(rk).sum(-1, keepdims=True) / D
                rk = np.stack([ora.fwht(r) for r in rk]) / D
                tol_k = half * np.abs(rk) + mag * (np.log2(D) + 1) * 2.0 ** -23 + 2.0 ** -25
            assert (np.abs(vd[:, h].double().cpu().numpy() - rv) <= tol_v).all()
            assert (np.abs(kd[:, h].double().cpu().numpy() - rk) <= tol_k).all()


def test_bad_entries_are_skipped():
    cache, _ = make_cache(2, 2, 128, 64, 4, 2, 64)
    k, v = tokens(20, 2, 128, "bf16", 1), tokens(20, 2, 128, "bf16", 2)
    good = [1, 16, 3, 16]
    cases = [([2, 0, 0, 1], kvq.KVQ_DEVERR_BAD_PAGE), ([-1, 0, 0, 1], kvq.KVQ_DEVERR_BAD_PAGE),
             ([0, 64, 0, 1], kvq.KVQ_DEVERR_CAPACITY), ([0, -1, 0, 1], kvq.KVQ_DEVERR_CAPACITY),
             ([0, 15, 0, 2], kvq.KVQ_DEVERR_CAPACITY), ([0, 0, 0, 17], kvq.KVQ_DEVERR_CAPACITY),
             ([0, 0, 0, -1], kvq.KVQ_DEVERR_CAPACITY), ([0, 0, -1, 1], kvq.KVQ_DEVERR_BAD_POS),
             ([0, 0, 20, 1], kvq.KVQ_DEVERR_BAD_POS), ([0, 0, 2 ** 31 - 1, 16], kvq.KVQ_DEVERR_BAD_POS)]
    want, _ = make_cache(2, 2, 128, 64, 4, 2, 64)
    kvq.kvq_quantize_append_ragged(want, k, v, i32([good]))
    for bad, flag in cases:
        for t in (cache.k_codes, cache.v_codes, cache.k_params, cache.v_params):
            t.zero_()
        slots = i32([bad, good, [0, 0, 0, 0]])
        kvq.kvq_quantize_append_ragged(cache, k, v, slots)
        assert kvq.kvq_device_error_flags() == flag, bad
        assert torch.equal(cache.k_codes, want.k_codes)
        assert torch.equal(cache.v_params, want.v_params)
        ko = torch.full((20, 2, 128), 7.0, device="cuda")
        vo = ko.clone()
        kvq.kvq_dequantize_ragged(cache, slots, 20, k_out=ko, v_out=vo)
        assert kvq.kvq_device_error_flags() == flag, bad
        named = torch.zeros(20, dtype=torch.bool)
        named[3:19] = True
        assert (ko[~named] == 7.0).all() and (vo[~named] == 7.0).all()
        assert (ko[named] != 7.0).any()


# ----------------------------------------------------------- chunk attention
def _chunk_case(lens, n_new, Hq, Hkv, D, bits, G, gv, P, rot, dtype, causal, seed=0, scale=0.0,
                out_dtype=None, tail=0, q_scale=1.0):
    B, cap = len(lens), (max(lens + [1]) + 511) // 256 * 256
    cache, users = make_cache(B, Hkv, D, cap, *bits, G, gv, rot, P, 3, want=lens)
    kd, vd, cu_kv = fill(cache, users, lens, seed, centre=0.5)
    cu = [0]
    for n in n_new:
        cu.append(cu[-1] + n)
    q = tokens(cu[-1] + tail, Hq, D, dtype, seed + 9) * q_scale
    out = torch.full(q.shape, 7.0, dtype=out_dtype or q.dtype, device="cuda")
    got = kvq.kvq_chunk_attention(cache, q, i32(cu), i32(lens), max(n_new), max(lens),
                                  causal=causal, sm_scale=scale, out=out)
    assert kvq.kvq_device_error_flags() == 0
    assert got is out
    assert (out[cu[-1]:] == 7.0).all()  # rows behind the last sequence
    want, tol = attention_reference(q[:cu[-1]], kd, vd, cu_kv, cu, lens, causal, scale, out.dtype,
                                    rot)
    assert_close(out[:cu[-1]], want, tol)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("bits", [(4, 2), (2, 2), (2, 4), (2, 8), (4, 4), (4, 8), (8, 2), (8, 4),
                                  (8, 8)])
def test_chunk_bits_and_types(bits, dtype):
    _chunk_case([70, 200, 33], [5, 70, 1], 8, 2, 128, bits, 64, 0, 32, False, dtype, True)


@pytest.mark.parametrize("D,G,gv", [(128, 32, 0), (128, 64, 0), (128, 128, 0), (128, 32, 64),
                                    (128, 32, 128), (128, 64, 128), (64, 32, 0), (64, 64, 0),
                                    (64, 32, 64)])
@pytest.mark.parametrize("rot", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("bits", [(4, 2), (2, 8), (8, 4)])
def test_chunk_groups(D, G, gv, rot, dtype, bits):
    _chunk_case([150, 40], [30, 40], 4, 2, D, bits, G, gv, 0, rot, dtype, True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1), (3, 1), (28, 4), (8, 8), (32, 2), (48, 4),
                                    (64, 1)])
def test_chunk_heads(Hq, Hkv, dtype):
    _chunk_case([90, 130, 17], [9, 33, 17], Hq, Hkv, 128, (4, 2), 64, 0, 64, False, dtype, True)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("P", [0, 32, 64, 256])
@pytest.mark.parametrize("lens,n_new", [
    ([1], [1]), ([2], [2]), ([127], [127]), ([128], [128]), ([129], [129]), ([255], [1]),
    ([256], [255]), ([257], [2]), ([1, 1, 1], [1, 0, 1]), ([0, 5, 0], [0, 3, 0]),
    ([640, 16, 15, 17, 31, 33], [3, 16, 1, 17, 2, 33]), ([1000], [64]), ([1025], [513])])
def test_chunk_lengths(lens, n_new, P, causal):
    _chunk_case(lens, n_new, 4, 2, 128, (4, 2), 64, 0, P, False, "bf16", causal)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
def test_chunk_rows_that_see_nothing(D, dtype):
    # more queries than cached positions: the first ones see nothing (o = 0)
    _chunk_case([0, 3, 40], [4, 7, 90], 4, 2, D, (4, 2), 32, 0, 32, False, dtype, True)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("lens,n_new", [([2500, 3000], [1, 1]), ([2500, 3000], [4, 4]),
                                        ([4000], [700]), ([1500] * 20, [1] * 19 + [257]),
                                        ([5000, 100], [0, 3])])
def test_chunk_long_rows(lens, n_new, dtype):
    _chunk_case(lens, n_new, 8, 2, 128, (4, 2), 64, 0, 64, False, dtype, True, tail=3)


@pytest.mark.parametrize("dtype,out_dtype", [("bf16", "f32"), ("f32", "bf16"), ("f16", "bf16"),
                                             ("f32", "f16"), ("f16", "f32")])
def test_chunk_output_types(dtype, out_dtype):
    _chunk_case([300, 50], [40, 50], 8, 2, 128, (8, 4), 64, 0, 32, True, dtype, True,
                out_dtype=DT[out_dtype], scale=0.2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_scale", [2.0 ** -120, 2.0 ** -30, 30.0, 2.0 ** 18])
def test_chunk_query_ranges(dtype, q_scale):
    """Queries far outside binary16's range, with the scale that undoes it."""
    scale = 128 ** -0.5 / q_scale if q_scale != 30.0 else 0.0
    _chunk_case([300, 50], [40, 5], 8, 2, 128, (8, 8), 64, 0, 32, False, dtype, True,
                scale=scale, q_scale=q_scale)


def test_chunk_masked_positions_may_hold_anything():
    """NaN and infinite parameters past a row's length never reach it."""
    cache, _ = make_cache(2, 2, 128, 512, 4, 2, 64)
    lens = [130, 77]
    kd, vd, cu_kv = fill(cache, None, lens, 3)
    for t, D in ((cache.k_params, 2), (cache.v_params, 2)):
        par = t.view(torch.float16).view(2, 2, 512, -1)
        for b, n in enumerate(lens):
            par[b, :, n:] = float("nan")
            par[b, :, n + 1::2] = float("inf")
    for dtype in ("bf16", "f32"):
        q = tokens(70, 4, 128, dtype, 4)
        for causal in (True, False):
            out = kvq.kvq_chunk_attention(cache, q, i32([0, 60, 70]), i32(lens), 60, 512,
                                          causal=causal)
            want, tol = attention_reference(q, kd, vd, cu_kv, [0, 60, 70], lens, causal, 0.0,
                                            q.dtype)
            assert_close(out, want, tol)


def test_chunk_largest_values():
    """Keys and values up to binary16's largest number stay finite."""
    cache, _ = make_cache(1, 1, 128, 128, 4, 2, 64)
    g = torch.Generator().manual_seed(5)
    x = (torch.rand(100, 1, 128, generator=g) * 2 - 1) * 65504.0
    x[:, :, 0], x[:, :, 1] = 65504.0, -65504.0
    x[:, :, 64], x[:, :, 65] = 65504.0, -65504.0
    x = x.cuda()
    _, _, slots = kvq.kvq_plan_append(cache, i32([0]), i32([100]), 100)
    kvq.kvq_quantize_append_ragged(cache, x, x, slots)
    kd, vd = kvq.kvq_dequantize_ragged(cache, slots, 100, torch.float32)
    for dtype in ("bf16", "f32"):
        q = tokens(50, 2, 128, dtype, 4)
        out = kvq.kvq_chunk_attention(cache, q, i32([0, 50]), i32([100]), 50, 100,
                                      sm_scale=1e-6, out_dtype=torch.float32)
        want, tol = attention_reference(q, kd, vd, [0, 100], [0, 50], [100], True, 1e-6,
                                        torch.float32)
        # a stored group whose largest value passes 65504 (by the rounding of
        # its scale and zero, 2^-11 of its range of 131008 each) may be held
        # at 65504: one more such step
        assert_close(out, want, tol + 131008 * 2.0 ** -10)


def test_chunk_device_errors():
    cache, users = make_cache(2, 2, 128, 256, 4, 2, 64, P=32, spare=1, want=[100, 60])
    fill(cache, users, [100, 60], 1)
    q = tokens(12, 4, 128, "bf16", 2)
    ok = kvq.kvq_chunk_attention(cache, q, i32([0, 6, 12]), i32([100, 60]), 6, 100)

    def run(cu, lens, max_q=6, max_len=100):
        out = torch.full_like(ok, 7.0)
        kvq.kvq_chunk_attention(cache, q, i32(cu), i32(lens), max_q, max_len, out=out)
        return out, kvq.kvq_device_error_flags()

    out, flags = run([0, 6, 12], [300, 60])                     # past max_seq_len: clamped
    assert flags == kvq.KVQ_DEVERR_SEQ_LEN and torch.equal(out, ok)
    out, flags = run([0, 6, 13], [100, 60])                     # past the packed tokens: skipped
    assert flags == kvq.KVQ_DEVERR_BAD_POS and torch.equal(out[:6], ok[:6])
    assert (out[6:] == 7.0).all()
    out, flags = run([0, 6, 12], [100, 60], max_q=5)            # more queries than announced
    assert flags == kvq.KVQ_DEVERR_BAD_POS and (out == 7.0).all()
    out, flags = run([6, 0, 6], [100, 60])                      # not ascending
    assert flags == kvq.KVQ_DEVERR_BAD_POS and (out[6:] == 7.0).all()
    out, flags = run([-3, 3, 6], [100, 60])
    assert flags == kvq.KVQ_DEVERR_BAD_POS and (out[:3] == 7.0).all()
    out, flags = run([0, 6, 12], [-5, 60])                      # nothing cached
    assert (out[:6] == 0.0).all() and torch.equal(out[6:], ok[6:])
    cache.block_table[0, 1] = 1000                              # outside the pool: not followed
    out, flags = run([0, 6, 12], [100, 60])
    assert flags == kvq.KVQ_DEVERR_BAD_PAGE and torch.equal(out[6:], ok[6:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_chunk_many_rows(dtype):
    """Thousands of rows, most of them idle."""
    r = random.Random(3)
    lens = [r.randint(0, 90) for _ in range(3000)]
    n_new = [min(n, r.choice([0, 0, 0, 1, 2])) for n in lens]
    _chunk_case(lens, n_new, 2, 1, 64, (4, 2), 32, 0, 32, False, dtype, True)


def test_chunk_workspace():
    lens = [3000, 40]
    cache, users = make_cache(2, 2, 128, 4096, 4, 2, 64, P=64, spare=1, want=lens)
    fill(cache, users, lens, 1)
    q, cu = tokens(40, 4, 128, "bf16", 2), i32([0, 20, 40])
    need = kvq.kvq_chunk_workspace_bytes(cache, 4, 40, 20, 3000)
    assert need > 0
    for ws in (torch.empty(need - 1, dtype=torch.uint8, device="cuda"),
               torch.empty(need + 16, dtype=torch.uint8, device="cuda")[8:]):
        with pytest.raises(kvq.KvqError) as e:
            kvq.kvq_chunk_attention(cache, q, cu, i32(lens), 20, 3000, workspace=ws)
        assert e.value.status == kvq.KVQ_ERR_WORKSPACE
    # whatever the workspace holds, and wherever it lies in a larger one
    big = torch.full((need + 64,), 0xff, dtype=torch.uint8, device="cuda")
    a = kvq.kvq_chunk_attention(cache, q, cu, i32(lens), 20, 3000, workspace=big[16:16 + need])
    b = kvq.kvq_chunk_attention(cache, q, cu, i32(lens), 20, 3000)
    assert torch.equal(a, b) and (big[:16] == 0xff).all() and (big[16 + need:] == 0xff).all()


def test_chunk_nothing_cached_and_bounds_of_zero():
    cache, _ = make_cache(2, 2, 128, 256, 4, 2, 64)
    q = tokens(5, 4, 128, "f16", 2)
    out = kvq.kvq_chunk_attention(cache, q, i32([0, 2, 5]), i32([0, 0]), 3, 0)
    assert kvq.kvq_device_error_flags() == 0 and (out == 0).all()
    out = torch.full_like(q, 7.0)
    kvq.kvq_chunk_attention(cache, q, i32([0, 2, 5]), i32([0, 0]), 0, 0, out=out)
    assert kvq.kvq_device_error_flags() == kvq.KVQ_DEVERR_BAD_POS and (out == 7.0).all()


def test_single_tokens_of_strided_queries():
    lens = [100, 1, 64]
    cache, users = make_cache(3, 2, 128, 256, 4, 2, 64, P=64, spare=1, want=lens)
    kd, vd, cu_kv = fill(cache, users, lens, 2)
    q = tokens(3, 12, 128, "bf16", 5)[:, 4:8]
    out = kvq.kvq_chunk_attention(cache, q, i32([0, 1, 2, 3]), i32(lens), 1, 100)
    want, tol = attention_reference(q, kd, vd, cu_kv, [0, 1, 2, 3], lens, True, 0.0, q.dtype)
    assert_close(out, want, tol)


def test_a_cache_whose_fields_change():
    """The descriptor that a cache keeps follows its fields and buffers."""
    cache, _ = make_cache(1, 2, 128, 64, 4, 2, 64)
    k, v = tokens(16, 2, 128, "bf16", 1), tokens(16, 2, 128, "bf16", 2)
    _, _, slots = kvq.kvq_plan_append(cache, i32([0]), i32([16]), 16)
    kvq.kvq_quantize_append_ragged(cache, k, v, slots)
    a, _ = kvq.kvq_dequantize_ragged(cache, slots, 16, torch.float32)
    cache.k_codes = torch.zeros_like(cache.k_codes)
    b, _ = kvq.kvq_dequantize_ragged(cache, slots, 16, torch.float32)
    assert not torch.equal(a, b)
    cache.rotate_keys = True
    c, _ = kvq.kvq_dequantize_ragged(cache, slots, 16, torch.float32)
    assert not torch.equal(b, c)


def test_chunk_shared_prefix_pages_and_strided_queries():
    cache, users = make_cache(2, 2, 128, 128, 4, 2, 64, P=32, spare=4, want=[96, 0])
    kd, vd, _ = fill(cache, users, [96, 0], 1)
    cache.block_table[1, :3] = cache.block_table[0, :3]
    wide = tokens(11, 8, 128, "bf16", 3)
    q = wide[:, 2:6]
    out = kvq.kvq_chunk_attention(cache, q, i32([0, 4, 11]), i32([96, 64]), 7, 96)
    want, tol = attention_reference(q, torch.cat([kd, kd]), torch.cat([vd, vd]), [0, 96],
                                    [0, 4, 11], [96, 64], True, 0.0, torch.bfloat16)
    assert_close(out, want, tol)


def test_chunk_is_the_same_every_time():
    """No atomics order the sums: equal bits on equal inputs."""
    cache, users = make_cache(3, 2, 128, 4096, 4, 2, 64, P=64, spare=1, want=[4000, 900, 30])
    fill(cache, users, [4000, 900, 30], 1)
    for dtype in ("bf16", "f16", "f32"):
        q = tokens(40, 8, 128, dtype, 5)
        outs = [kvq.kvq_chunk_attention(cache, q, i32([0, 4, 34, 40]), i32([4000, 900, 30]), 30,
                                        4000) for _ in range(3)]
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_single_tokens_agree_with_decode():
    lens = [1, 700, 64, 2000]
    cache, users = make_cache(4, 2, 128, 2048, 4, 2, 64, P=64, spare=1, want=lens)
    kd, vd, cu_kv = fill(cache, users, lens, 2)
    for dtype in ("bf16", "f16", "f32"):
        q = tokens(4, 8, 128, dtype, 5)
        a = kvq.kvq_chunk_attention(cache, q, i32([0, 1, 2, 3, 4]), i32(lens), 1, 2000)
        want, tol = attention_reference(q, kd, vd, cu_kv, [0, 1, 2, 3, 4], lens, True, 0.0,
                                        q.dtype)
        assert_close(a, want, tol)
        # idle rows and single tokens, by the general path
        b = kvq.kvq_chunk_attention(cache, q[:3].contiguous(), i32([0, 1, 1, 2, 3]), i32(lens),
                                    1, 2000)
        q3, cu3 = q[:3], [0, 1, 1, 2, 3]
        want, tol = attention_reference(q3, kd, vd, cu_kv, cu3, lens, True, 0.0, q.dtype)
        assert_close(b, want, tol)


# ------------------------------------------------------------- all together
class _Model:
    """Host mirror of the cached values of every row."""

    def __init__(self, B):
        self.k = [[] for _ in range(B)]
        self.v = [[] for _ in range(B)]


@pytest.mark.parametrize("P,dtype,rot", [(64, "bf16", False), (32, "f16", True), (0, "f32", False)])
def test_serving_steps(P, dtype, rot):
    """Prefill chunks, single tokens, draft tokens and their rejection, a row
    that finishes and one that takes its place: pages planned, tokens appended
    and attended, every step against the reference."""
    r = random.Random(7)
    B, Hkv, Hq, D, cap = 5, 2, 8, 128, 512
    lens = [0] * B
    cache, users = make_cache(B, Hkv, D, cap, 4, 2, 64, 0, rot, P, 0, want=[cap] * B)
    vals = _Model(B)
    for step in range(8):
        old = list(lens)
        new = []
        for b in range(B):
            kind = r.choice(["one", "draft", "chunk", "idle"])
            add = {"one": 1, "draft": 4, "chunk": r.randint(2, 90), "idle": 0}[kind]
            new.append(min(cap, old[b] + add))
        if step == 4:
            new[2] = old[2]
        total = sum(n - o for o, n in zip(old, new))
        got, cu, slots = kvq.kvq_plan_append(cache, i32(old), i32(new), total, users)
        assert got.tolist() == new
        k = tokens(total, Hkv, D, dtype, 100 + step, 1.0, 0.5)
        v = tokens(total, Hkv, D, dtype, 200 + step)
        q = tokens(total, Hq, D, dtype, 300 + step)
        kvq.kvq_quantize_append_ragged(cache, k, v, slots)
        kd, vd = kvq.kvq_dequantize_ragged(cache, slots, total, torch.float32)
        c = cu.tolist()
        for b in range(B):
            vals.k[b].append(kd[c[b]:c[b + 1]])
            vals.v[b].append(vd[c[b]:c[b + 1]])
        out = kvq.kvq_chunk_attention(cache, q, cu, got, max(1, max(n - o for o, n in zip(old, new))),
                                      max(new))
        allk = [torch.cat(x) for x in vals.k]
        allv = [torch.cat(x) for x in vals.v]
        at = [0]
        for x in allk:
            at.append(at[-1] + x.shape[0])
        want, tol = attention_reference(q, torch.cat(allk), torch.cat(allv), at, c, new, True, 0.0,
                                        q.dtype, rot)
        assert_close(out, want, tol)
        # some draft tokens are rejected, row 2 finishes in step 4
        back = [max(o, n - r.randint(0, 3)) if n - o == 4 else n for o, n in zip(old, new)]
        if step == 4:
            back[2] = 0
        lens_t, _, _ = kvq.kvq_plan_append(cache, got, i32(back), 0, users)
        lens = lens_t.tolist()
        assert lens == back
        for b in range(B):
            vals.k[b] = [torch.cat(vals.k[b])[:lens[b]]]
            vals.v[b] = [torch.cat(vals.v[b])[:lens[b]]]
        if P:
            assert int(users.sum()) == sum((n + P - 1) // P for n in lens)
    assert kvq.kvq_device_error_flags() == 0


def test_step_in_a_cuda_graph():
    """Plan, append, read-back and attention captured once and replayed with
    other lengths and tokens; two graphs share one workspace."""
    B, Hkv, Hq, D, T = 4, 2, 8, 128, 40
    cache, users = make_cache(B, Hkv, D, 1024, 4, 2, 64, P=32, spare=0, want=[1024] * B)
    kd, vd, cu_kv = fill(cache, users, [600, 900, 31, 64], 1)
    old, new = i32([600, 900, 31, 64]), i32([600, 900, 31, 64])
    k, v, q = (torch.zeros(T, h, D, dtype=torch.bfloat16, device="cuda") for h in (Hkv, Hkv, Hq))
    need = kvq.kvq_chunk_workspace_bytes(cache, Hq, T, T, 1024)
    ws = torch.empty(max(16, need), dtype=torch.uint8, device="cuda")

    def step():
        lens, cu, slots = kvq.kvq_plan_append(cache, old, new, T, users)
        kvq.kvq_quantize_append_ragged(cache, k, v, slots)
        out = kvq.kvq_chunk_attention(cache, q, cu, lens, T, 1024, workspace=ws)
        return lens, cu, slots, out

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs, results = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            results.append(step())
        graphs.append(g)
    lens = [600, 900, 31, 64]
    vals = [kd[cu_kv[b]:cu_kv[b + 1]] for b in range(B)], [vd[cu_kv[b]:cu_kv[b + 1]] for b in range(B)]
    for i, add in enumerate(([1, 1, 1, 1], [30, 0, 1, 9], [0, 4, 36, 0])):
        nxt = [n + a for n, a in zip(lens, add)]
        old.copy_(i32(lens))
        new.copy_(i32(nxt))
        k.copy_(tokens(T, Hkv, D, "bf16", 10 + i))
        v.copy_(tokens(T, Hkv, D, "bf16", 20 + i))
        q.copy_(tokens(T, Hq, D, "bf16", 30 + i))
        graphs[i % 2].replay()
        got, cu, slots, out = results[i % 2]
        a, w = kvq.kvq_dequantize_ragged(cache, slots, T, torch.float32)
        c = cu.tolist()
        assert got.tolist() == nxt and c[-1] == sum(add)
        for x, y in zip(vals, (a, w)):
            for b in range(B):
                x[b] = torch.cat([x[b], y[c[b]:c[b + 1]]])
        at = [0]
        for x in vals[0]:
            at.append(at[-1] + x.shape[0])
        want, tol = attention_reference(q[:c[-1]], torch.cat(vals[0]), torch.cat(vals[1]), at, c, nxt,
                                        True, 0.0, torch.bfloat16)
        assert_close(out[:c[-1]], want, tol)
        lens = nxt
    assert kvq.kvq_device_error_flags() == 0


def test_calls_on_another_stream():
    cache, users = make_cache(2, 2, 128, 512, 4, 2, 64, P=32, spare=1, want=[300, 80])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    k, v = tokens(380, 2, 128, "bf16", 1), tokens(380, 2, 128, "bf16", 2)
    q = tokens(20, 4, 128, "bf16", 3)
    s.wait_stream(torch.cuda.current_stream())
    lens, cu, slots = kvq.kvq_plan_append(cache, i32([0, 0]), i32([300, 80]), 380, users, stream=s)
    kvq.kvq_quantize_append_ragged(cache, k, v, slots, stream=s)
    a, b = kvq.kvq_dequantize_ragged(cache, slots, 380, torch.float32, stream=s)
    out = kvq.kvq_chunk_attention(cache, q, i32([0, 10, 20]), lens, 10, 300, stream=s)
    s.synchronize()
    want, tol = attention_reference(q, a, b, [0, 300], [0, 10, 20], [300, 80], True, 0.0, q.dtype)
    assert_close(out, want, tol)


def test_two_calls_at_once():
    """Two streams, each with its own cache and workspace, many calls each."""
    def make(seed, dtype):
        cache, users = make_cache(3, 2, 128, 2048, 4, 2, 64, P=64, spare=1, want=[2000, 300, 77])
        kd, vd, cu_kv = fill(cache, users, [2000, 300, 77], seed)
        q = tokens(90, 8, 128, dtype, seed + 5)
        return cache, q, attention_reference(q, kd, vd, cu_kv, [0, 60, 64, 90], [2000, 300, 77], True,
                                             0.0, q.dtype)

    cases = [make(1, "bf16"), make(2, "f32")]
    cu, lens = i32([0, 60, 64, 90]), i32([2000, 300, 77])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[], []]
    for _ in range(4):
        for i, (cache, q, _) in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                outs[i].append(kvq.kvq_chunk_attention(cache, q, cu, lens, 60, 2000))
    torch.cuda.synchronize()
    assert kvq.kvq_device_error_flags() == 0
    for (_, _, (want, tol)), got in zip(cases, outs):
        for o in got:
            assert_close(o, want, tol)
            assert torch.equal(o, got[0])


def test_cache_beyond_32_bit_offsets():
    """A pool whose code arrays pass 4 GiB: its last pages are written, read
    back and attended like the first ones."""
    P, pages = 256, 16900
    free = torch.cuda.mem_get_info()[0]
    if free < 30 << 30:
        pytest.skip("not enough device memory")
    table = torch.tensor([[pages - 1, 3, pages - 2]], dtype=torch.int32)
    cache = kvq.KVCache.allocate(1, 8, 128, 3 * P, 8, 8, 64, page_size=P, num_pages=pages,
                                 block_table=table)
    assert cache.k_codes.numel() > 2 ** 32
    small = kvq.KVCache.allocate(1, 8, 128, 3 * P, 8, 8, 64)
    T = 700
    k, v = tokens(T, 8, 128, "bf16", 1), tokens(T, 8, 128, "bf16", 2)
    q = tokens(65, 16, 128, "bf16", 3)
    outs = []
    for c in (cache, small):
        users = torch.zeros(pages, dtype=torch.int32, device="cuda") if c.page_size else None
        if users is not None:
            users[table[0].long()] = 1  # the pages are the row's already
        _, _, slots = kvq.kvq_plan_append(small, i32([0]), i32([T]), T)
        if c.page_size:
            m = slots.cpu()
            m[:, 0] = table[0][(m[:, 1] // P).long()] * (m[:, 3] > 0)
            m[:, 1] %= P
            slots = m.cuda()
        kvq.kvq_quantize_append_ragged(c, k, v, slots)
        a, b = kvq.kvq_dequantize_ragged(c, slots, T, torch.float32)
        outs.append((a, b, kvq.kvq_chunk_attention(c, q, i32([0, 65]), i32([T]), 65, T)))
    assert kvq.kvq_device_error_flags() == 0
    for x, y in zip(*outs):
        assert torch.equal(x, y)


def test_python_refusals():
    cache, users = make_cache(2, 2, 128, 64, 4, 2, 64, P=32, spare=1, want=[64, 64])
    z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    i2, i3 = z(2, dt=torch.int32), z(3, dt=torch.int32)
    x, q, slots = z(4, 2, 128), z(4, 4, 128), z(4, 4, dt=torch.int32)
    bad = [
        lambda: kvq.kvq_plan_append(cache, i2, i2, 4),                       # no user counts
        lambda: kvq.kvq_plan_append(cache, i3, i2, 4, users),
        lambda: kvq.kvq_plan_append(cache, i2.long(), i2, 4, users),
        lambda: kvq.kvq_plan_append(cache, i2, i2, 4, users[:1]),
        lambda: kvq.kvq_plan_append(cache, i2.cpu(), i2, 4, users),
        lambda: kvq.kvq_quantize_append_ragged(cache, x, x[:3], slots),
        lambda: kvq.kvq_quantize_append_ragged(cache, x, x.half(), slots),
        lambda: kvq.kvq_quantize_append_ragged(cache, q, q, slots),          # other heads
        lambda: kvq.kvq_quantize_append_ragged(cache, x.double(), x.double(), slots),
        lambda: kvq.kvq_quantize_append_ragged(cache, x, x, slots.view(-1)),
        lambda: kvq.kvq_quantize_append_ragged(cache, x, x, slots.t().contiguous().t()),
        lambda: kvq.kvq_quantize_append_ragged(cache, q[:, ::2], q[:, ::2], slots),
        lambda: kvq.kvq_dequantize_ragged(cache, slots, 4, torch.float64),
        lambda: kvq.kvq_dequantize_ragged(cache, slots, 4, k_out=x),
        lambda: kvq.kvq_dequantize_ragged(cache, slots, 5, k_out=x, v_out=x),
        lambda: kvq.kvq_chunk_attention(cache, q, i2, i2, 4, 64),
        lambda: kvq.kvq_chunk_attention(cache, q, i3, i3, 4, 64),
        lambda: kvq.kvq_chunk_attention(cache, q[0], i3, i2, 4, 64),
        lambda: kvq.kvq_chunk_attention(cache, q, i3, i2, 4, 64, out=x),
        lambda: kvq.kvq_chunk_attention(cache, z(4, 3, 128), i3, i2, 4, 64),
    ]
    for call in bad:
        with pytest.raises((ValueError, kvq.KvqError)):
            call()
    # nothing to do
    none = z(0, 4, 128)
    assert kvq.kvq_chunk_attention(cache, none, i3, i2, 4, 64).shape == (0, 4, 128)
    kvq.kvq_quantize_append_ragged(cache, x[:0], x[:0], slots)
    assert kvq.kvq_device_error_flags() == 0
