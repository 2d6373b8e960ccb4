"""GPU tests of how the serving step is called: on which stream a call's
memory lives, from several host threads, with padded batches, with values that
are not finite, and with waits that run out."""
import ctypes
import threading
import time

import pytest
import torch

import kv_cache_mixed_kvq_b200 as kvq
from tests.serve_util import (assert_close, attention_reference, fill, i32, make_cache, tokens)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- streams
def _stream_of(t):
    """Raw stream that the caching allocator took a tensor's memory on."""
    at = t.data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= at < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the allocator's memory")


def test_results_and_workspace_belong_to_the_call_stream(monkeypatch):
    lens = [3000, 40]
    cache, users = make_cache(2, 2, 128, 4096, 4, 2, 64, P=64, spare=4, want=lens)
    fill(cache, users, lens, 1)
    q, q2 = tokens(40, 4, 128, "bf16", 2), tokens(2, 4, 128, "bf16", 2)
    k, v = tokens(2, 2, 128, "bf16", 3), tokens(2, 2, 128, "bf16", 4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    made = []
    empty = torch.empty

    def logged(*a, **kw):
        made.append(empty(*a, **kw))
        return made[-1]

    monkeypatch.setattr(torch, "empty", logged)
    with torch.cuda.stream(s):
        old, new, cu, at = i32(lens), i32([3001, 41]), i32([0, 20, 40]), i32([3000, 40])
    plan = kvq.kvq_plan_append(cache, old, new, 2, users, stream=s)
    kvq.kvq_quantize_append_ragged(cache, k, v, plan[2], stream=s)
    results = [*plan, *kvq.kvq_dequantize_ragged(cache, plan[2], 2, stream=s),
               kvq.kvq_chunk_attention(cache, q, cu, at, 20, 3000, stream=s),
               kvq.kvq_decode_attention(cache, q2, at, 3000, stream=s)]
    kn = k.view(2, 2, 1, 128)
    results.append(kvq.kvq_append_decode_attention(cache, kn, kn, q2, plan[0], 3001, stream=s))
    monkeypatch.undo()
    assert len(made) >= 9  # (results and three workspaces)
    for t in made + results:
        assert _stream_of(t) == s.cuda_stream
    s.synchronize()
    assert kvq.kvq_device_error_flags() == 0


def test_overlapping_calls_by_the_stream_argument():
    """Calls on two streams from one current stream, which takes and drops
    memory of the workspaces' size in between: each has its own memory."""
    lens, cu = [2000, 300, 77], i32([0, 60, 64, 90])

    def make(seed, dtype):
        cache, users = make_cache(3, 2, 128, 2048, 4, 2, 64, P=64, spare=1, want=lens)
        kd, vd, cu_kv = fill(cache, users, lens, seed)
        q = tokens(90, 8, 128, dtype, seed + 5)
        want = attention_reference(q, kd, vd, cu_kv, [0, 60, 64, 90], lens, True, 0.0, q.dtype)
        return cache, q, want

    cases = [make(1, "bf16"), make(2, "f32")]
    need = max(kvq.kvq_chunk_workspace_bytes(c, 8, 90, 60, 2000) for c, _, _ in cases)
    assert need > 0
    at = i32(lens)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[], []]
    for _ in range(6):
        for i, (cache, q, _) in enumerate(cases):
            outs[i].append(kvq.kvq_chunk_attention(cache, q, cu, at, 60, 2000, stream=streams[i]))
            torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert kvq.kvq_device_error_flags() == 0
    for (_, _, (want, tol)), got in zip(cases, outs):
        for o in got:
            assert_close(o, want, tol)
            assert torch.equal(o, got[0])


def test_arguments_may_be_dropped_after_the_call():
    """Memory of the current stream that a call on another one still reads is
    not given out again."""
    cache, _ = make_cache(1, 2, 128, 256, 4, 2, 64)
    slots = kvq.kvq_plan_append(cache, i32([0]), i32([200]), 200)[2]
    k, v = tokens(200, 2, 128, "bf16", 1), tokens(200, 2, 128, "bf16", 2)
    kvq.kvq_quantize_append_ragged(cache, k, v, slots)
    want = [t.clone() for t in (cache.k_codes, cache.v_codes)]
    for t in (cache.k_codes, cache.v_codes):
        t.zero_()
    s = torch.cuda.Stream()
    k2, v2 = k.clone(), v.clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)  # some 10 ms before the call's turn
    kvq.kvq_quantize_append_ragged(cache, k2, v2, slots, stream=s)
    size = k2.numel()
    del k2, v2
    for _ in range(4):
        torch.full((size,), 9.0, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    assert torch.equal(cache.k_codes, want[0]) and torch.equal(cache.v_codes, want[1])


# ------------------------------------------------- values that are not finite
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rot", [False, True])
@pytest.mark.parametrize("lens,n_new", [([150, 70], [40, 3]), ([300], [200]),
                                        ([3000, 40], [3, 40]), ([4000], [300])])
def test_query_that_is_not_finite(lens, n_new, rot, dtype):
    """NaN in its own rows of the output, whole units (narrow and wide) and
    divided ones; the other rows as ever."""
    cache, users = make_cache(len(lens), 2, 128, 4096, 4, 2, 64, 0, rot, 64, 3, want=lens)
    kd, vd, cu_kv = fill(cache, users, lens, 1)
    cu = [0]
    for n in n_new:
        cu.append(cu[-1] + n)
    q = tokens(cu[-1], 8, 128, dtype, 9)
    want, tol = attention_reference(q, kd, vd, cu_kv, cu, lens, True, 0.0, q.dtype, rot)
    bad = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    for t, h, d, x in ((0, 0, 5, NAN), (1, 7, 0, INF), (cu[-1] - 1, 3, 127, -INF),
                       (cu[-1] // 2, 4, 64, NAN)):
        q[t, h, d] = x
        bad[t, h] = True
    q[2, 1] = NAN
    bad[2, 1] = True
    out = kvq.kvq_chunk_attention(cache, q, i32(cu), i32(lens), max(n_new), max(lens))
    assert kvq.kvq_device_error_flags() == 0
    assert torch.isnan(out[bad]).all()
    assert_close(out[~bad], want[~bad], tol[~bad])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("L,n,t", [(200, 60, 150), (3000, 4, 2997), (3000, 4, 17), (700, 300, 640)])
def test_visible_key_that_is_not_finite(L, n, t, dtype):
    """A NaN scale of a key reaches the queries that see it, and no other."""
    cache, _ = make_cache(1, 2, 128, 4096, 4, 2, 64)
    kd, vd, cu_kv = fill(cache, None, [L], 1)
    cache.k_params.view(torch.float16).view(2, 4096, 2, 2)[1, t, 0, 0] = NAN
    q = tokens(n, 8, 128, dtype, 9)
    want, tol = attention_reference(q, kd, vd, cu_kv, [0, n], [L], True, 0.0, q.dtype)
    out = kvq.kvq_chunk_attention(cache, q, i32([0, n]), i32([L]), n, L)
    bad = torch.zeros(n, 8, dtype=torch.bool, device="cuda")
    bad[max(0, t - (L - n)):, 4:] = True
    assert torch.isnan(out[bad]).all()
    assert_close(out[~bad], want[~bad], tol[~bad])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("L", [1, 1000])
def test_scores_of_minus_infinity_alone(L, dtype):
    """0 / 0, not the output of a query that sees nothing."""
    cache, _ = make_cache(1, 1, 128, 1024, 4, 2, 64)
    fill(cache, None, [L], 1)
    par = cache.k_params.view(torch.float16).view(1024, 2, 2)
    par[:, :, 0], par[:, :, 1] = 0.0, -INF
    q = tokens(2, 1, 128, dtype, 9).abs() + 0.5
    out = kvq.kvq_chunk_attention(cache, q, i32([0, 2]), i32([L]), 2, L, causal=False)
    assert torch.isnan(out).all()
    none = kvq.kvq_chunk_attention(cache, q, i32([0, 2]), i32([0]), 2, L, causal=False)
    assert (none == 0).all()


# ------------------------------------------------------- sums past 32 bits
def _plan_only(B, cap, P=0, pages=0, table=None):
    """A cache for planning alone, which touches no codes or parameters."""
    bufs = [torch.zeros(64, dtype=torch.uint8, device="cuda") for _ in range(4)]
    return kvq.KVCache(B, 1, 64, cap, 2, 2, 64, *bufs, page_size=P, num_pages=pages,
                       block_table=table)


def _summed(new):
    cu = [0]
    for n in new:
        cu.append(min(cu[-1] + n, 2 ** 31 - 1))
    return cu


def test_plan_of_more_tokens_and_tiles_than_32_bits_count():
    new = [70] + [2 ** 30] * 40 + [9]
    lens, cu, m = kvq.kvq_plan_append(_plan_only(42, 2 ** 30), i32([0] * 42), i32(new), 100)
    assert kvq.kvq_device_error_flags() == kvq.KVQ_DEVERR_CAPACITY
    assert lens.tolist() == new and cu.tolist() == _summed(new)
    got = [e for e in m.tolist() if e[3]]
    assert got == [[0, 16 * i, 16 * i, min(16, 70 - 16 * i)] for i in range(5)] + \
        [[1, 0, 70, 16], [1, 16, 86, 14]]


def test_plan_of_refused_tokens_past_32_bits():
    """Rows that the pool cannot serve keep their place in cu_tokens."""
    P, B = 2 ** 20, 4
    table = torch.full((B, 1024), -1, dtype=torch.int32, device="cuda")
    users = torch.zeros(3, dtype=torch.int32, device="cuda")
    new = [2 ** 30, 2 ** 30, 2 ** 30, 5]
    lens, cu, m = kvq.kvq_plan_append(_plan_only(B, 2 ** 30, P, 3, table), i32([0] * B), i32(new),
                                      5, users)
    assert kvq.kvq_device_error_flags() == kvq.KVQ_DEVERR_CAPACITY | kvq.KVQ_DEVERR_NO_PAGE
    assert lens.tolist() == [0] * B and cu.tolist() == _summed(new)
    assert (m == 0).all() and (users == 0).all() and (table == -1).all()


@pytest.mark.parametrize("pages", [1000, 20000])
def test_plan_of_more_pages_than_32_bits_count(pages):
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("not enough device memory")
    B, P, cap = 8192, 32, 2 ** 24
    table = torch.full((B, cap // P), -1, dtype=torch.int32, device="cuda")
    users = torch.zeros(pages, dtype=torch.int32, device="cuda")
    users[::3] = 1
    new = [150, 0, 40] + [cap] * (B - 4) + [33]  # (the last row comes after the sum has passed 2^31)
    lens, cu, m = kvq.kvq_plan_append(_plan_only(B, cap, P, pages, table), i32([0] * B), i32(new),
                                      190, users)
    assert kvq.kvq_device_error_flags() == kvq.KVQ_DEVERR_CAPACITY | kvq.KVQ_DEVERR_NO_PAGE
    assert lens.tolist() == [150, 0, 40] + [0] * (B - 3) and cu.tolist() == _summed(new)
    assert table[0, :5].tolist() == [1, 2, 4, 5, 7] and table[2, :2].tolist() == [8, 10]
    assert int((table >= 0).sum()) == 7 and int((users != 0).sum()) == (pages + 2) // 3 + 7
    got = [e for e in m.tolist() if e[3]]
    assert len(got) == 10 + 3 and sum(e[3] for e in got) == 190
    assert got[-1] == [10, 0, 182, 8]


# ------------------------------------------------------- several host threads
def test_threads_plan_batches_of_different_sizes():
    """The kernel's shared-memory limit is the function's, not a thread's."""
    lib, ready, statuses = kvq.library(), threading.Barrier(6), []

    def prepare(B):
        cache, old, new = _plan_only(B, 64), i32([0] * B), i32([1] * B)
        lens, cu = torch.empty_like(old), i32([0] * (B + 1))
        m = torch.empty(B, 4, dtype=torch.int32, device="cuda")
        s = torch.cuda.Stream()
        args = (ctypes.byref(cache.desc()), old.data_ptr(), new.data_ptr(), B, None,
                lens.data_ptr(), cu.data_ptr(), m.data_ptr(), B, s.cuda_stream)
        return args, (cache, old, new, lens, cu, m, s)

    jobs = [prepare(B) for B in (8192, 4500, 8000, 5000, 7000, 4200)]
    torch.cuda.synchronize()

    def work(args):
        ready.wait()
        statuses.append({lib.kvq_plan_append(*args) for _ in range(3000)})

    threads = [threading.Thread(target=work, args=(args,)) for args, _ in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert statuses == [{kvq.KVQ_OK}] * 6
    for _, (_, _, new, lens, cu, _, _) in jobs:
        assert torch.equal(lens, new) and cu[-1].item() == new.numel()
    assert kvq.kvq_device_error_flags() == 0


# -------------------------------------------------------- launches in a chain
@pytest.mark.parametrize("schedule", ["splits", "balanced"])
def test_attention_right_after_the_plan_that_writes_its_lengths(schedule, monkeypatch):
    """The decode kernel may start while the planner still runs: it reads the
    lengths only after it, with either division of the work."""
    if schedule == "balanced":
        monkeypatch.setenv("KVQ_DECODE_SCHEDULE", "balanced")
    B, P, cap, pages = 64, 32, 1024, 1 << 20  # (many pages: the planner takes its time)
    planned = _plan_only(B, cap, P, pages, torch.full((B, cap // P), -1, dtype=torch.int32,
                                                      device="cuda"))
    users = torch.ones(pages, dtype=torch.int32, device="cuda")
    users[-30000:] = 0
    cache, _ = make_cache(B, 1, 64, cap, 4, 2, 64)
    fill(cache, None, [cap] * B, 1)
    q, none = tokens(B, 4, 64, "bf16", 3), i32([0] * B)
    steps = [i32([1 + (37 * b + 211 * i) % cap for b in range(B)]) for i in range(12)]
    want = [kvq.kvq_decode_attention(cache, q, new, cap) for new in steps]
    torch.cuda.synchronize()
    got = []
    for new in steps:
        lens = kvq.kvq_plan_append(planned, none, new, B * cap, users)[0]
        got.append(kvq.kvq_decode_attention(cache, q, lens, cap))
    torch.cuda.synchronize()
    assert kvq.kvq_device_error_flags() == 0
    for x, y in zip(got, want):
        assert torch.equal(x, y)


# ------------------------------------------------- padded and idle single tokens
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("P,rot,Hq", [(0, False, 8), (64, False, 14), (64, True, 8), (0, True, 32)])
@pytest.mark.parametrize("long", [False, True])
def test_single_tokens_of_padded_steps(long, P, rot, Hq, dtype):
    """As many packed tokens as rows, but some rows idle: each token goes with
    its own row, and the padding behind the last one is left as it was."""
    lens = [100, 3000, 64, 1, 2111, 0] if long else [100, 130, 64, 1, 33, 0]
    cache, users = make_cache(6, 2, 128, 4096, 4, 2, 64, 0, rot, P, 3, want=lens)
    kd, vd, cu_kv = fill(cache, users, lens, 1)
    q = tokens(6, Hq, 128, dtype, 9)
    for cu in ([0, 1, 1, 2, 3, 3, 4], [0, 0, 1, 1, 1, 2, 2], [0, 1, 2, 3, 4, 5, 6], [0] * 7):
        out = torch.full_like(q, 7.0)
        kvq.kvq_chunk_attention(cache, q, i32(cu), i32(lens), 1, max(lens), out=out)
        assert kvq.kvq_device_error_flags() == 0
        n = cu[-1]
        assert (out[n:] == 7.0).all()
        if n:
            want, tol = attention_reference(q[:n], kd, vd, cu_kv, cu, lens, True, 0.0, q.dtype, rot)
            assert_close(out[:n], want, tol)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("long", [False, True])
def test_single_tokens_with_unusable_offsets(long, dtype):
    lens = [3000, 40, 9] if long else [200, 40, 9]
    cache, users = make_cache(3, 2, 128, 4096, 4, 2, 64, 0, False, 64, 3, want=lens)
    kd, vd, cu_kv = fill(cache, users, lens, 1)
    q = tokens(3, 8, 128, dtype, 9)
    want, tol = attention_reference(q, kd, vd, cu_kv, [0, 1, 2, 3], lens, True, 0.0, q.dtype)
    # the rows that are served, by offsets with a fault in another row
    for cu, served in (([0, 1, 3, 3], [0]), ([0, 1, 2, 2 ** 31 - 1], [0, 1]), ([0, 1, 1, 0], [0]),
                       ([2, 3, 4, 4], None), ([-1, 0, 1, 2], None)):
        out = torch.full_like(q, 7.0)
        kvq.kvq_chunk_attention(cache, q, i32(cu), i32(lens), 1, max(lens), out=out)
        assert kvq.kvq_device_error_flags() == kvq.KVQ_DEVERR_BAD_POS, cu
        if served is not None:
            n = len(served)
            assert_close(out[:n], want[:n], tol[:n])
            assert (out[n:] == 7.0).all()


@pytest.mark.parametrize("P", [0, 64])
@pytest.mark.parametrize("Hq,Hkv", [(8, 4), (32, 4), (20, 4)])
def test_rotated_f16_single_tokens_keep_their_query(Hq, Hkv, P):
    """Scores in the hundreds of two positions that nearly tie: a query rounded
    to one binary16 would move the weights by 0.01 and more.  The same rows by
    the decode kernel (as many tokens as rows) and by the tile kernel."""
    B, D = 96, 128
    lens = [2 + b % 2 for b in range(B)]
    cache, users = make_cache(B, Hkv, D, 128, 8, 8, 32, 0, True, P, 1, want=lens)
    kd, vd, cu_kv = fill(cache, users, lens, 1)
    q = tokens(B, Hq, D, "f16", 9) * 128.0
    cu = list(range(B + 1))
    want, tol = attention_reference(q, kd, vd, cu_kv, cu, lens, True, 0.0, torch.float32, True)
    # The largest weight of a row is held at 1 or more in binary16, whose
    # smallest step is 2^-24: a weight less than that part of the largest (the
    # scores differ by hundreds) may vanish, at most 3 of them, each moving the
    # output by |v| times as much.
    tol = tol + 3 * 2.0 ** -24 * vd.abs().max().item()
    out = kvq.kvq_chunk_attention(cache, q, i32(cu), i32(lens), 1, 3, out_dtype=torch.float32)
    assert_close(out, want, tol)
    cu[-1] = B - 1  # the last row idle, its token not there
    out = kvq.kvq_chunk_attention(cache, q[:-1], i32(cu), i32(lens), 1, 3, out_dtype=torch.float32)
    assert_close(out, want[:-1], tol[:-1])
    assert kvq.kvq_device_error_flags() == 0


# --------------------------------------------------- the ends of binary16's range
@pytest.mark.parametrize("D,bits", [(128, (4, 2)), (64, (2, 8)), (128, (8, 4))])
@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_largest_values_in_two_halves(dtype, D, bits):
    """Groups whose stored scale and zero pass 65504 by their roundings are held
    to 2^-22 like all others where keys and values have two binary16 halves."""
    cache, _ = make_cache(1, 1, D, 128, *bits, 64)
    g = torch.Generator().manual_seed(5)
    x = (torch.rand(100, 1, D, generator=g) * 2 - 1) * 65504.0
    x[:, :, 0::64], x[:, :, 1::64] = 65504.0, -65504.0 + 16.0 * torch.arange(100).view(100, 1, 1)
    x = x.cuda()
    _, _, slots = kvq.kvq_plan_append(cache, i32([0]), i32([100]), 100)
    kvq.kvq_quantize_append_ragged(cache, x, x, slots)
    kd, vd = kvq.kvq_dequantize_ragged(cache, slots, 100, torch.float32)
    assert max(kd.max().item(), vd.max().item()) > 65504.0
    q = tokens(50, 2, D, dtype, 4)
    out = kvq.kvq_chunk_attention(cache, q, i32([0, 50]), i32([100]), 50, 100, sm_scale=1e-6,
                                  out_dtype=torch.float32)
    want, tol = attention_reference(q, kd, vd, [0, 100], [0, 50], [100], True, 1e-6, torch.float32)
    assert_close(out, want, tol)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("which", ["scale", "zero"])
def test_visible_value_that_is_infinite(which, dtype):
    """Infinite parameters are not brought back into range."""
    cache, _ = make_cache(1, 1, 128, 256, 4, 4, 64)
    L, t = 200, 130
    kd, vd, cu_kv = fill(cache, None, [L], 1)
    cache.v_params.view(torch.float16).view(256, 2, 2)[t, 1, int(which == "zero")] = INF
    q = tokens(20, 4, 128, dtype, 9)
    want, tol = attention_reference(q, kd, vd, cu_kv, [0, 20], [L], False, 0.0, q.dtype)
    out = kvq.kvq_chunk_attention(cache, q, i32([0, 20]), i32([L]), 20, L, causal=False)
    assert_close(out[..., :64], want[..., :64], tol[..., :64])
    assert not torch.isfinite(out[..., 64:]).any()


# ------------------------------------------------------------ failure detection
@pytest.mark.parametrize("dtype,D,bits", [("bf16", 128, (4, 2)), ("bf16", 128, (8, 8)),
                                          ("f16", 128, (4, 2)), ("f32", 64, (2, 4))])
@pytest.mark.parametrize("lens,n_new", [([200, 90], [60, 2]), ([3000, 40], [4, 40]),
                                        ([2000], [700])])
@pytest.mark.parametrize("drop_stage", [0, 1])
def test_chunk_wait_that_runs_out(drop_stage, lens, n_new, dtype, D, bits):
    """One ring block of the first CTA never fills up: the launch flags it and
    ends, with products of other tiles or none in flight, and the next call is
    as ever.  (No fault and no hang: every wait is bounded, here to 1 ms.)"""
    cache, users = make_cache(len(lens), 2, D, 4096, *bits, 32, 0, False, 64, 3, want=lens)
    fill(cache, users, lens, 1)
    cu = [0]
    for n in n_new:
        cu.append(cu[-1] + n)
    q, at, offsets = tokens(cu[-1], 8, D, dtype, 9), i32(lens), i32(cu)
    bytes_before = [t.clone() for t in (cache.k_codes, cache.v_codes, cache.k_params)]

    def run():
        out = kvq.kvq_chunk_attention(cache, q, offsets, at, max(n_new), max(lens))
        torch.cuda.synchronize()
        return out

    ref = run()
    assert kvq.kvq_last_device_error() == 0
    kvq.kvq_debug_inject_wait_timeout(drop_stage, wait_limit_ns=1_000_000)
    t0 = time.perf_counter()
    run()
    elapsed = time.perf_counter() - t0
    assert kvq.kvq_last_device_error() == kvq.KVQ_DEVERR_TIMEOUT
    assert elapsed < 0.5
    for t, before in zip((cache.k_codes, cache.v_codes, cache.k_params), bytes_before):
        assert torch.equal(t, before)
    assert torch.equal(run(), ref) and kvq.kvq_last_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [40, 1500])
def test_rows_that_overlap(n, dtype):
    """Offsets that go back leave rows that name the same tokens: as much work as
    there are rows, whatever num_tokens says.  Nothing is attended then."""
    B, lens = 7, [1600] * 7
    cache, users = make_cache(B, 2, 64, 2048, 4, 2, 64, P=64, spare=1, want=lens)
    kd, vd, cu_kv = fill(cache, users, lens, 1)
    q = tokens(n, 4, 64, dtype, 2)
    out = torch.full_like(q, 7.0)
    kvq.kvq_chunk_attention(cache, q, i32([0, n, 0, n, 0, n, 0, n]), i32(lens), n, 1600, out=out)
    assert kvq.kvq_device_error_flags() == kvq.KVQ_DEVERR_BAD_POS
    assert (out == 7.0).all()
    # one step back, and no overlap: the usable row is served
    cu = [n, n, n, 0, n, n, n, n]
    kvq.kvq_chunk_attention(cache, q, i32(cu), i32(lens), n, 1600, out=out)
    assert kvq.kvq_device_error_flags() == kvq.KVQ_DEVERR_BAD_POS
    want, tol = attention_reference(q, kd, vd, cu_kv, [0, 0, 0, 0, n, n, n, n], lens, True, 0.0,
                                    q.dtype)
    assert_close(out, want, tol)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tile_attention_right_after_the_plan(dtype):
    """Offsets and lengths that the kernel before writes, by the tile kernel."""
    B, P, cap, pages = 64, 32, 1024, 1 << 20
    planned = _plan_only(B, cap, P, pages, torch.full((B, cap // P), -1, dtype=torch.int32,
                                                      device="cuda"))
    users = torch.ones(pages, dtype=torch.int32, device="cuda")
    users[-3000:] = 0
    cache, _ = make_cache(B, 1, 64, cap, 4, 2, 64)
    fill(cache, None, [cap] * B, 1)
    q = tokens(3 * B, 4, 64, dtype, 3)
    steps = []
    for i in range(12):
        old = [32 * ((7 * b + 5 * i) % 31) for b in range(B)]
        steps.append((i32(old), i32([n + 1 + (b + i) % 3 for b, n in enumerate(old)])))
    want = []
    for old, new in steps:
        cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
        cu[1:] = (new - old).cumsum(0)
        want.append((int(cu[-1]), kvq.kvq_chunk_attention(cache, q, cu, new, 3, cap)))
    torch.cuda.synchronize()
    got = []
    for old, new in steps:
        lens, cu, _ = kvq.kvq_plan_append(planned, old, new, 3 * B, users)
        got.append(kvq.kvq_chunk_attention(cache, q, cu, lens, 3, cap))
    torch.cuda.synchronize()
    assert kvq.kvq_device_error_flags() == 0
    for x, (n, y) in zip(got, want):
        assert torch.equal(x[:n], y[:n])


def test_append_right_after_the_plan_and_the_read_back():
    """A prefix moved to another cache: plan, read-back and append in a chain,
    each reading what the one before writes."""
    T, H, D = 700, 2, 128
    a, _ = make_cache(1, H, D, 1024, 8, 8, 32)
    kd, vd, _ = fill(a, None, [T], 1)
    moved, _ = make_cache(1, H, D, 1024, 4, 2, 64)
    slots = kvq.kvq_plan_append(a, i32([0]), i32([T]), T)[2]
    kvq.kvq_quantize_append_ragged(moved, kd, vd, slots)
    want = [t.clone() for t in (moved.k_codes, moved.v_codes, moved.k_params, moved.v_params)]
    old, new = i32([0]), i32([T])
    ko, vo = torch.zeros_like(kd), torch.zeros_like(vd)
    for _ in range(8):
        for t in (moved.k_codes, moved.v_codes, moved.k_params, moved.v_params):
            t.zero_()
        ko.zero_(), vo.zero_()
        slots = kvq.kvq_plan_append(moved, old, new, T)[2]
        kvq.kvq_dequantize_ragged(a, slots, T, k_out=ko, v_out=vo)
        kvq.kvq_quantize_append_ragged(moved, ko, vo, slots)
        for t, w in zip((moved.k_codes, moved.v_codes, moved.k_params, moved.v_params), want):
            assert torch.equal(t, w)
    assert kvq.kvq_device_error_flags() == 0


@pytest.mark.parametrize("env", [("KVQ_DECODE_KERNEL", "tcgen05"), ("KVQ_SPLIT_TOKENS", "64"),
                                 ("KVQ_DECODE_SCHEDULE", "balanced")])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_padded_single_tokens_with_the_decode_settings(env, dtype, monkeypatch):
    """The opt-in kernel and schedule do not look rows up: they are not taken."""
    monkeypatch.setenv(*env)
    lens = [100, 3000, 64, 1, 2111, 0]
    cache, users = make_cache(6, 2, 128, 4096, 4, 2, 64, 0, False, 64, 3, want=lens)
    kd, vd, cu_kv = fill(cache, users, lens, 1)
    q, cu = tokens(6, 16, 128, dtype, 9), [0, 1, 2, 2, 3, 4, 4]
    out = torch.full_like(q, 7.0)
    kvq.kvq_chunk_attention(cache, q, i32(cu), i32(lens), 1, max(lens), out=out)
    assert kvq.kvq_device_error_flags() == 0 and (out[4:] == 7.0).all()
    want, tol = attention_reference(q[:4], kd, vd, cu_kv, cu, lens, True, 0.0, q.dtype)
    assert_close(out[:4], want, tol)


def test_captured_calls_on_the_capture_stream_by_argument():
    """stream= inside a capture: the results are the graph's memory."""
    lens = [1500, 40]
    cache, users = make_cache(2, 2, 128, 2048, 4, 2, 64, P=64, spare=1, want=lens)
    fill(cache, users, lens, 1)
    q, cu, at = tokens(40, 4, 128, "bf16", 2), i32([0, 20, 40]), i32(lens)
    want = kvq.kvq_chunk_attention(cache, q, cu, at, 20, 1500)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out = kvq.kvq_chunk_attention(cache, q, cu, at, 20, 1500, stream=s)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert kvq.kvq_device_error_flags() == 0
