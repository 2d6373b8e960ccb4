"""Measured cases of the serving-step operators: page and slot-map planning,
ragged quantize-append with read-back, and attention of a chunk of new tokens
over the packed (paged) cache.

A serving step over a ragged batch is, per layer, "append the step's new keys
and values, then let the new queries attend to everything cached", with the
pages and the map of destinations planned once for all layers:

  plan    kvq_plan_append: from the rows' old and new lengths, pages are taken
          from (or returned to) the pool, the block table is updated, and the
          slot map is written: one entry (block, position, first token, count)
          per 16-position tile that receives tokens;
  append  kvq_quantize_append_ragged: the packed new tokens [total][Hkv][D]
          are quantized into the tiles of the slot map; the pass then reads
          them back with kvq_dequantize_ragged, so that what the cache holds
          in 2, 4 or 8 bits is compared as the values it stands for;
  chunk   kvq_chunk_attention: ragged queries [total][Hq][D] against the
          packed cache; query i of the n_b queries of row b attends to
          positions [0, len_b - n_b + i] (causal) or [0, len_b).

`run` computes either the plain form (elementary torch operations in 32 bits)
or, where `own` is true, the calls of kv_cache_mixed_kvq_b200.
"""
import math
import random

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
DEV = "cuda"


# ------------------------------------------------------------------- cases
def listed():
    gqa = dict(q_heads=32, kv_heads=8, head_dim=128, group=64, group_v=0, rotate=False)
    k4v2 = dict(bits_k=4, bits_v=2, dtype="bf16")
    return [
        # one decode step of 64 ragged requests: every row grows by one token,
        # a few of them into a new page; then the step is rolled back (the
        # smallest call of the planner: latency)
        dict(name="plan_decode_step", op="plan", batch=64, page=64, cap=8192, lo=512, hi=8191,
             grow_lo=1, grow_hi=1, spare=512, lens_seed=1),
        # a large mixed step: 1000 requests, each with up to 257 new tokens
        # (prefill chunks, draft tokens, some rows idle), pages of 32
        dict(name="plan_mixed_1000", op="plan", batch=1000, page=32, cap=8192, lo=0, hi=7900,
             grow_lo=0, grow_hi=257, spare=9000, lens_seed=2),
        # a decode step's write: one new token for each of 64 requests
        dict(name="append_decode_step", op="append", batch=64, page=64, cap=8192, lo=512, hi=8191,
             grow_lo=1, grow_hi=1, lens_seed=3, **gqa, **k4v2),
        # a prefill step's write: 16 ragged chunks, about 8200 tokens
        dict(name="append_chunks", op="append", batch=16, page=128, cap=4096, lo=0, hi=2048,
             grow_lo=9, grow_hi=1015, lens_seed=4, **gqa, **k4v2),
        # binary32 inputs, head_dim 64, rotated keys, finer key groups, odd
        # lengths, slot layout (no pages)
        dict(name="append_f32_rotated", op="append", batch=5, page=0, cap=2048, lo=1, hi=777,
             grow_lo=101, grow_hi=1201, lens_seed=5, q_heads=8, kv_heads=4, head_dim=64, group=32,
             group_v=64, rotate=True, bits_k=8, bits_v=4, dtype="f32"),
        # verification of 4 draft tokens for each of 16 requests
        dict(name="chunk_verify_4", op="chunk", batch=16, page=64, cap=8192, lo=512, hi=8000,
             grow_lo=4, grow_hi=4, first=0, causal=True, lens_seed=6, **gqa, **k4v2),
        # the form for single tokens: a decode step of 64 ragged requests
        dict(name="chunk_single_token", op="chunk", batch=64, page=64, cap=8192, lo=512, hi=8191,
             grow_lo=1, grow_hi=1, first=0, causal=True, lens_seed=7, **gqa, **k4v2),
        # one 2048-token chunk deep in a long context (chunked prefill)
        dict(name="chunk_2048_at_24576", op="chunk", batch=1, page=256, cap=32768, lo=24576,
             hi=24576, grow_lo=2048, grow_hi=2048, first=0, causal=True, lens_seed=8, **gqa,
             **k4v2),
        # prefill from an empty cache: ragged prompts of 2000 to 4000 tokens
        dict(name="chunk_prefill_ragged", op="chunk", batch=4, page=128, cap=4096, lo=0, hi=0,
             grow_lo=2000, grow_hi=4000, first=0, causal=True, lens_seed=9, **gqa, **k4v2),
        # a mixed step, 7 query heads per kv head: one chunk of 257 tokens
        # among 15 requests that decode one token each
        dict(name="chunk_mixed_28q4", op="chunk", batch=16, page=64, cap=4096, lo=200, hi=3800,
             grow_lo=1, grow_hi=1, first=257, causal=True, lens_seed=10, q_heads=28, kv_heads=4,
             head_dim=128, group=64, group_v=128, rotate=False, bits_k=2, bits_v=4, dtype="f16"),
        # not causal (a block of tokens refined together), 8-bit keys, rotated,
        # slot layout
        dict(name="chunk_full_k8v4", op="chunk", batch=3, page=0, cap=4096, lo=1000, hi=3500,
             grow_lo=100, grow_hi=333, first=0, causal=False, lens_seed=11, q_heads=32, kv_heads=8,
             head_dim=128, group=32, group_v=32, rotate=True, bits_k=8, bits_v=4, dtype="bf16"),
        # binary32 queries and output, single head, head_dim 64, odd lengths
        dict(name="chunk_f32_d64", op="chunk", batch=2, page=32, cap=1024, lo=0, hi=500,
             grow_lo=17, grow_hi=131, first=0, causal=True, lens_seed=12, q_heads=4, kv_heads=2,
             head_dim=64, group=32, group_v=0, rotate=False, bits_k=4, bits_v=2, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    seed = rng.randrange(1 << 20)
    op = rng.choice(["plan", "append", "chunk", "chunk"])
    page = rng.choice([0, 32, 64, 128, 256])
    head_dim = rng.choice([64, 128, 128])
    group = rng.choice([32, 64, 128] if head_dim == 128 else [32, 64])
    group_v = rng.choice([0] + [g for g in (64, 128) if group < g <= head_dim])
    heads = rng.choice([(1, 1), (4, 2), (8, 8), (28, 4), (32, 8), (48, 4)])
    shape = dict(q_heads=heads[0], kv_heads=heads[1], head_dim=head_dim, group=group,
                 group_v=group_v, rotate=rng.random() < 0.25, bits_k=rng.choice([2, 4, 8]),
                 bits_v=rng.choice([2, 4, 8]), dtype=rng.choice(["bf16", "bf16", "f16", "f32"]))
    if op == "plan":
        batch = _log_int(rng, 1, 1000)
        hi = _log_int(rng, 1, 7900)
        return dict(op="plan", batch=batch, page=rng.choice([32, 64, 128]), cap=8192,
                    lo=rng.randint(0, hi), hi=hi, grow_lo=0, grow_hi=_log_int(rng, 1, 280),
                    spare=0, lens_seed=seed)
    if op == "append":
        batch = _log_int(rng, 1, 64)
        grow_hi = _log_int(rng, 1, max(1, min(2000, 16000 // batch)))
        grow_lo = rng.choice([0, rng.randint(1, grow_hi)])  # 0: some rows idle
        return dict(op="append", batch=batch, page=page, cap=4096, lo=0, hi=_log_int(rng, 1, 2048),
                    grow_lo=grow_lo, grow_hi=grow_hi, first=0 if grow_lo else grow_hi,
                    lens_seed=seed, **shape)
    batch = _log_int(rng, 1, 32)
    # at most as many scores as the largest listed case
    hi = _log_int(rng, 1, 6000)
    grow_hi = max(1, min(2000, _log_int(rng, 1, max(2, int(4e8 / (batch * (hi + 600) * heads[0]))))))
    grow_lo = rng.choice([0, 1, grow_hi, rng.randint(1, grow_hi)])  # 0: some rows idle
    return dict(op="chunk", batch=batch, page=page, cap=8192, lo=rng.randint(0, hi), hi=hi,
                grow_lo=grow_lo, grow_hi=grow_hi, first=0 if grow_lo else grow_hi,
                causal=rng.random() < 0.8, lens_seed=seed, **shape)


def _lens(case):
    """(old, new) lengths of the rows: part of the case, not of the seed."""
    r = random.Random(case["lens_seed"])
    old = [r.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]
    grow = [r.randint(case["grow_lo"], case["grow_hi"]) for _ in range(case["batch"])]
    if case.get("first"):
        grow[0] = case["first"]
    new = [min(case["cap"], o + g) for o, g in zip(old, grow)]
    return old, new


def _group_v(case):
    return case["group_v"] or case["group"]


def _row_bytes(case):
    """Bytes of one position of one kv head in the packed cache."""
    D = case["head_dim"]
    return D * (case["bits_k"] + case["bits_v"]) / 8 + 4 * (D / case["group"] + D / _group_v(case))


def work(case):
    old, new = _lens(case)
    total = sum(n - o for o, n in zip(old, new))
    if case["op"] == "plan":
        P = case["page"]
        took = sum((n + P - 1) // P - (o + P - 1) // P for o, n in zip(old, new))
        pool = sum((o + P - 1) // P for o in old) + took + case["spare"]
        tiles = sum((n + 15) // 16 - o // 16 for o, n in zip(old, new) if n > o)
        # reserve: lengths in, lengths and offsets out, the pool's user counts
        # read, a table and a count word per page taken, the map's tiles out;
        # roll back: lengths in, lengths and offsets out, a table and a count
        # word per page returned
        return {"bytes": 2 * 16 * case["batch"] + 4 * pool + 2 * 8 * took + 16 * tiles,
                "flops": 0}
    D, Hkv, es = case["head_dim"], case["kv_heads"], 4 if case["dtype"] == "f32" else 2
    if case["op"] == "append":
        # tokens in, packed rows out; packed rows in, values out
        return {"bytes": total * Hkv * (2 * 2 * D * es + 2 * _row_bytes(case)),
                "flops": total * Hkv * 2 * D * 6}
    cached = sum(new) * Hkv * _row_bytes(case)
    pairs = sum((n - o) * (o + n + 1) // 2 if case["causal"] else (n - o) * n
                for o, n in zip(old, new))
    return {"bytes": cached + 2 * total * case["q_heads"] * D * es,
            "flops": 4.0 * pairs * case["q_heads"] * D}


# --------------------------------------------------- cache format in torch
def _k_place(D, b):
    """Byte and shift of the code of element d inside a K row."""
    d = np.arange(D)
    E = 16 // b
    bit = 16 * (d % 2) + b * ((d // 8) % E)
    return (d % 8) // 2 * (D * b // 32) + 4 * ((d // 8) // E) + bit // 8, bit % 8


def _v_place(D, b):
    """Byte and shift of the code of (position k, element d) in a V tile."""
    k, d = np.arange(16)[:, None], np.arange(D)[None, :]
    E, W = 16 // b, D * b // 128
    N = D * b // 16
    P = min(16, N)
    lane = 4 * (d % 8) + (k % 8) // 2
    bit = 16 * (k % 2) + b * ((d // 8) % E)
    n = 4 * ((k // 8) * W + (d // 8) // E) + bit // 8
    return (n // P) * 32 * P + lane * P + n % P, bit % 8


def _on(a, dtype=torch.int64):
    return torch.as_tensor(np.ascontiguousarray(a), dtype=dtype, device=DEV)


def _pack_tables(D, b):
    """For K rows: the 8/b elements of each byte; for V tiles: the bytes of
    each position and the elements of each of them (low bits first)."""
    off, sh = _k_place(D, b)
    order = np.lexsort((sh, off))
    k_elem = order.reshape(D * b // 8, 8 // b)
    off, sh = _v_place(D, b)
    v_byte = np.empty((16, D * b // 8), np.int64)
    v_elem = np.empty((16, D * b // 8, 8 // b), np.int64)
    for k in range(16):
        order = np.lexsort((sh[k], off[k])).reshape(D * b // 8, 8 // b)
        v_elem[k], v_byte[k] = order, off[k][order[:, 0]]
    return k_elem, v_byte, v_elem


def _hadamard(x):
    """Butterfly h = 1, 2, ..., D/2 over the last axis, each step one sum."""
    D = x.shape[-1]
    h = 1
    while h < D:
        y = x.reshape(x.shape[:-1] + (D // (2 * h), 2, h))
        x = torch.stack((y[..., 0, :] + y[..., 1, :], y[..., 0, :] - y[..., 1, :]), -2)
        x = x.reshape(x.shape[:-3] + (D,))
        h *= 2
    return x


def _quantize(x, bits, group):
    """Codes (uint8) and binary16 (scale, zero) of x [..., D] in binary32."""
    g = x.reshape(x.shape[:-1] + (x.shape[-1] // group, group))
    mn, mx = g.amin(-1, keepdim=True) + 0.0, g.amax(-1, keepdim=True) + 0.0
    # (by a tensor: a quotient by a number may be taken as a product)
    scale = (mx - mn) / torch.full_like(mx, float(2 ** bits - 1))
    inv = torch.ones_like(scale) / scale
    flat = (scale == 0) | ~torch.isfinite(scale) | ~torch.isfinite(inv)
    codes = torch.round((g - mn) * torch.where(flat, 0.0, inv)).clamp(0, 2 ** bits - 1)
    codes = torch.where(flat, 0.0, codes).to(torch.uint8).reshape(x.shape)
    return codes, torch.cat((scale, mn), -1).to(torch.float16)


def _bytes_of(codes, elem, b):
    """Packs codes [..., D] through the element table [..., bytes, 8/b]."""
    c = codes[..., elem] if elem.dim() == 2 else \
        torch.gather(codes, -1, elem.reshape(elem.shape[0], 1, -1).expand(
            -1, codes.shape[1], -1)).reshape(codes.shape[:2] + elem.shape[1:])
    sh = torch.arange(0, 8, b, device=c.device)
    return (c.to(torch.int32) << sh).sum(-1).to(torch.uint8)


def _write(s, k, v, block, pos):
    """Quantizes k, v [n][Hkv][D] into positions `pos` of blocks `block`."""
    c = s["case"]
    bk, bv = c["bits_k"], c["bits_v"]
    k, v = k.float(), v.float()
    if c["rotate"]:
        k = _hadamard(k)
    kc, kp = _quantize(k, bk, c["group"])
    vc, vp = _quantize(v, bv, _group_v(c))
    s["k_codes"][block, :, pos] = _bytes_of(kc, s["k_elem"], bk)
    s["k_params"][block, :, pos] = kp
    s["v_params"][block, :, pos] = vp
    r = pos % 16
    h = torch.arange(c["kv_heads"], device=DEV)
    s["v_codes"][block[:, None, None], h[None, :, None], (pos // 16)[:, None, None],
                 s["v_byte"][r][:, None, :]] = _bytes_of(vc, s["v_elem"][r], bv)


def _read(s, block, pos):
    """Values (binary32) of K (in its stored basis) and V at the positions."""
    c = s["case"]
    kc = s["k_codes"][block, :, pos][..., s["k_off"]].to(torch.int32) >> s["k_sh"]
    r = pos % 16
    h = torch.arange(c["kv_heads"], device=DEV)
    vc = s["v_codes"][block[:, None, None], h[None, :, None], (pos // 16)[:, None, None],
                      s["v_off"][r][:, None, :]].to(torch.int32) >> s["v_sh"][r][:, None, :]

    def values(code, bits, par, group):
        par = par.float().repeat_interleave(group, -2)
        return (code & (2 ** bits - 1)).float() * par[..., 0] + par[..., 1]

    return (values(kc, c["bits_k"], s["k_params"][block, :, pos], c["group"]),
            values(vc, c["bits_v"], s["v_params"][block, :, pos], _group_v(c)))


# ------------------------------------------------------------------ prepare
def _pages(case, old, new, seed):
    """Block table [B][cap / P] for lengths `old` and the pages' user counts,
    scattered over the pool as after many allocations; room to grow to `new`."""
    P, B = case["page"], case["batch"]
    have = [(o + P - 1) // P for o in old]
    want = [(n + P - 1) // P for n in new]
    pool = max(1, sum(want) + case.get("spare", 0))
    order = np.random.default_rng(seed).permutation(pool)
    table = np.full((B, case["cap"] // P), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :have[b]] = order[at:at + have[b]]
        at += have[b]
    users = np.zeros(pool, np.int32)
    users[order[:at]] = 1
    return table, users, order[at:], have, want


def _token_places(case, table, old, new):
    """(block, position in it) of each packed new token, and the slot map."""
    P = case["page"] or case["cap"]
    block, pos, entries, token = [], [], [], 0
    for b, (o, n) in enumerate(zip(old, new)):
        p = np.arange(o, n)
        blk = table[b, p // P] if case["page"] else np.full(p.shape, b)
        block.append(blk)
        pos.append(p % P)
        q = o
        while q < n:
            e = min(n, q // 16 * 16 + 16)
            entries.append((blk[q - o], q % P, token, e - q))
            token += e - q
            q = e
    total = sum(n - o for o, n in zip(old, new))
    m = np.zeros((min(total, total // 16 + 2 * case["batch"]), 4), np.int32)
    if entries:
        m[:len(entries)] = entries
    cat = lambda a: np.concatenate(a) if a else np.zeros(0, np.int64)  # noqa: E731
    return cat(block).astype(np.int64), cat(pos).astype(np.int64), m


def prepare(case, seed):
    old, new = _lens(case)
    s = dict(case=case, old=_on(old, torch.int32), new=_on(new, torch.int32))
    cu = np.concatenate(([0], np.cumsum(np.array(new) - np.array(old))))
    s["total"], s["cu"] = int(cu[-1]), _on(cu, torch.int32)
    if case["op"] == "plan":
        table, users, _, _, _ = _pages(case, old, new, seed)
        s["table"], s["users"] = _on(table, torch.int32), _on(users, torch.int32)
        s["entries"] = min(s["total"], s["total"] // 16 + 2 * case["batch"])
        if own:
            import kv_cache_mixed_kvq_b200 as kvq
            # (the planner touches no codes: one-layer buffers of one head)
            s["cache"] = kvq.KVCache.allocate(
                case["batch"], 1, 64, case["cap"], 2, 2, 64, page_size=case["page"],
                num_pages=users.size, block_table=s["table"])
        return s

    # the cache's arrays, by block: a page, or a row's slot
    D, Hkv, bk, bv = case["head_dim"], case["kv_heads"], case["bits_k"], case["bits_v"]
    P = case["page"] or case["cap"]
    table = None
    if case["page"]:
        table, _, spare, have, want = _pages(case, old, new, seed)
        at = 0
        for b in range(case["batch"]):
            table[b, have[b]:want[b]] = spare[at:at + want[b] - have[b]]
            at += want[b] - have[b]
    blocks = int(sum(want)) if case["page"] else case["batch"]
    blocks = max(1, blocks)
    s.update(
        k_codes=torch.zeros((blocks, Hkv, P, D * bk // 8), dtype=torch.uint8, device=DEV),
        v_codes=torch.zeros((blocks, Hkv, P // 16, 2 * D * bv), dtype=torch.uint8, device=DEV),
        k_params=torch.zeros((blocks, Hkv, P, D // case["group"], 2), dtype=torch.float16,
                             device=DEV),
        v_params=torch.zeros((blocks, Hkv, P, D // _group_v(case), 2), dtype=torch.float16,
                             device=DEV),
        table=_on(table, torch.int32) if table is not None else None)
    off, sh = _k_place(D, bk)
    s["k_off"], s["k_sh"] = _on(off), _on(sh, torch.int32)
    off, sh = _v_place(D, bv)
    s["v_off"], s["v_sh"] = _on(off), _on(sh, torch.int32)
    s["k_elem"] = _on(_pack_tables(D, bk)[0])
    s["v_byte"], s["v_elem"] = (_on(t) for t in _pack_tables(D, bv)[1:])
    block, pos, m = _token_places(case, table, old, new)
    s["block"], s["pos"], s["map"] = _on(block), _on(pos), _on(m, torch.int32)

    # keys with per-channel centres and a few outlier channels, normal values
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    rnd = lambda *shape: torch.randn(shape, generator=g, device=DEV)  # noqa: E731
    centre, mult = 2.0 * rnd(Hkv, D), torch.ones((Hkv, D), device=DEV)
    mult.scatter_(1, rnd(Hkv, D).argsort(-1)[:, :max(1, round(0.02 * D))], 10.0)
    dt = DT[case["dtype"]]

    def tokens(n):
        return ((centre + rnd(n, Hkv, D)) * mult).to(dt), rnd(n, Hkv, D).to(dt)

    if case["op"] == "append":
        s["k"], s["v"] = tokens(s["total"])
    else:
        # fill every cached position, a few thousand tokens at a time
        block, pos, _ = _token_places(case, table, [0] * len(new), new)
        for i in range(0, len(block), 8192):
            k, v = tokens(len(block[i:i + 8192]))
            _write(s, k, v, _on(block[i:i + 8192]), _on(pos[i:i + 8192]))
        s["q"] = rnd(s["total"], case["q_heads"], D).to(dt)
        s["max_q"] = max(n - o for o, n in zip(old, new))
        s["max_len"] = max(new)
        # plain form: each row's queries padded to max_q, cached positions of
        # each row by (block, position)
        n_b = np.array(new) - np.array(old)
        i = np.arange(s["max_q"])[None, :]
        s["pad"] = _on(np.minimum(cu[:-1, None] + np.minimum(i, np.maximum(n_b[:, None], 1) - 1),
                                  s["total"] - 1))
        s["limit"] = _on(np.minimum(np.array(old)[:, None] + i + 1, np.array(new)[:, None])
                         if case["causal"] else np.array(new)[:, None] + 0 * i)
        tok_row = np.repeat(np.arange(len(new)), n_b)
        s["tok_row"], s["tok_i"] = _on(tok_row), _on(np.arange(s["total"]) - cu[tok_row])
    if own:
        import kv_cache_mixed_kvq_b200 as kvq
        buf = [s[n].reshape(-1).view(torch.uint8)
               for n in ("k_codes", "v_codes", "k_params", "v_params")]
        s["cache"] = kvq.KVCache(case["batch"], Hkv, D, case["cap"], bk, bv, case["group"], *buf,
                                 rotate_keys=case["rotate"], group_v=case["group_v"],
                                 page_size=case["page"],
                                 num_pages=blocks if case["page"] else 0, block_table=s["table"])
        if case["op"] == "chunk":
            need = kvq.kvq_chunk_workspace_bytes(s["cache"], case["q_heads"], s["total"],
                                                 s["max_q"], s["max_len"])
            s["workspace"] = torch.empty(need, dtype=torch.uint8, device=DEV) if need else None
    return s


# --------------------------------------------------------------------- run
def _plan_plain(s, old, new, total, entries):
    """One planning call on the state's table and user counts (both updated
    in place); rows are served in order, free pages in ascending order."""
    c, table, users = s["case"], s["table"], s["users"]
    P, B = c["page"], c["batch"]
    old, new = old.long(), new.long()
    have, want = (old + P - 1) // P, (new + P - 1) // P
    j = torch.arange(table.shape[1], device=DEV)[None, :]
    # return the pages past the new lengths
    back = (j >= want[:, None]) & (j < have[:, None])
    extra = torch.zeros(users.numel() + 1, dtype=torch.int32, device=DEV)
    extra.index_add_(0, torch.where(back, table.long(), users.numel()).reshape(-1),
                     back.reshape(-1).int())
    users -= extra[:-1]
    table.masked_fill_(back, -1)
    # take the free pages in order
    need = (want - have).clamp(min=0)
    upto = need.cumsum(0)
    free = users == 0
    rank = torch.where(free, free.cumsum(0) - 1, users.numel())
    row = torch.searchsorted(upto, rank, right=True)
    take = row < B
    row = row.clamp(max=B - 1)
    at = row * table.shape[1] + have[row] + rank - (upto - need)[row]
    flat = torch.cat((table.reshape(-1), table.new_zeros(1)))
    flat[torch.where(take, at, table.numel())] = torch.arange(
        users.numel(), dtype=torch.int32, device=DEV)
    table.copy_(flat[:-1].reshape(table.shape))
    users += take.int()
    # offsets and the slot map
    n = (new - old).clamp(min=0)
    cu = torch.cat((n.new_zeros(1), n.cumsum(0)))
    tiles = torch.where(n > 0, (new + 15) // 16 - old // 16, 0)
    end = tiles.cumsum(0)
    e = torch.arange(entries, device=DEV)
    row = torch.searchsorted(end, e, right=True)
    live = row < B
    row = row.clamp(max=B - 1)
    tile = old[row] // 16 + e - (end - tiles)[row]
    first = torch.maximum(tile * 16, old[row])
    last = torch.minimum(tile * 16 + 16, new[row])
    page = table[row, (tile * 16 // P).clamp(0, table.shape[1] - 1)].long()
    m = torch.stack((page, first % P, cu[row] + first - old[row], last - first), -1)
    return new.int(), cu.int(), torch.where(live[:, None], m, 0).int()


def _attend_plain(s):
    c = s["case"]
    P, D, Hkv, B = c["page"] or c["cap"], c["head_dim"], c["kv_heads"], c["batch"]
    T = (s["max_len"] + 15) // 16 * 16
    p = torch.arange(T, device=DEV)
    if c["page"]:
        block = s["table"].long()[:, p // P].clamp(min=0)
    else:
        block = torch.arange(B, device=DEV)[:, None].expand(B, T)
    k, v = _read(s, block.reshape(-1), (p % P).repeat(B))
    k = k.reshape(B, T, Hkv, D).permute(0, 2, 3, 1)
    v = v.reshape(B, T, Hkv, D).permute(0, 2, 1, 3)
    q = s["q"].float()
    if c["rotate"]:
        q = _hadamard(q) / D
    n, gq = s["max_q"], c["q_heads"] // Hkv
    q = q[s["pad"]].reshape(B, n, Hkv, gq, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * gq, D)
    x = (q @ k) * (1.0 / math.sqrt(D))
    masked = p[None, None, :] >= s["limit"][:, :, None]
    x = x.reshape(B, Hkv, n, gq, T).masked_fill_(masked[:, None, :, None, :], -math.inf)
    x = x - x.amax(-1, keepdim=True).clamp(min=-3e38)
    x = x.exp_()
    total = x.sum(-1, keepdim=True)
    v = torch.where((p[None, :] < s["new"][:, None])[:, None, :, None], v, 0.0)
    o = x.reshape(B, Hkv, n * gq, T) @ v
    o = o.reshape(B, Hkv, n, gq, D) / torch.where(total > 0, total, 1.0)
    o = o.permute(0, 2, 1, 3, 4).reshape(B, n, c["q_heads"], D)[s["tok_row"], s["tok_i"]]
    return o.to(DT[c["dtype"]])


def run(s):
    c = s["case"]
    if own:
        import kv_cache_mixed_kvq_b200 as kvq
    if c["op"] == "plan":
        # the step's pages are reserved, then returned as if all of its tokens
        # had been rejected
        if own:
            cache, users = s["cache"], s["users"]
            lens, cu, m = kvq.kvq_plan_append(cache, s["old"], s["new"], s["total"],
                                              page_users=users)
            back, none, _ = kvq.kvq_plan_append(cache, s["new"], s["old"], 0, page_users=users)
            table = cache.block_table
        else:
            lens, cu, m = _plan_plain(s, s["old"], s["new"], s["total"], s["entries"])
            back, none, _ = _plan_plain(s, s["new"], s["old"], 0, 0)
            table, users = s["table"], s["users"]
        return dict(lens=lens, cu=cu, map=m, back=back, none=none, table=table, users=users)
    if c["op"] == "append":
        dt = DT[c["dtype"]]
        if own:
            kvq.kvq_quantize_append_ragged(s["cache"], s["k"], s["v"], s["map"])
            k, v = kvq.kvq_dequantize_ragged(s["cache"], s["map"], s["total"], dt)
        else:
            _write(s, s["k"], s["v"], s["block"], s["pos"])
            k, v = _read(s, s["block"], s["pos"])
            if c["rotate"]:
                k = _hadamard(k) / c["head_dim"]
            k, v = k.to(dt), v.to(dt)
        return dict(k=k, v=v, k_params=s["k_params"], v_params=s["v_params"])
    if own:
        return kvq.kvq_chunk_attention(s["cache"], s["q"], s["cu"], s["new"], s["max_q"],
                                       s["max_len"], causal=c["causal"],
                                       workspace=s["workspace"])
    return _attend_plain(s)


# ------------------------------------------------------------------- exact
def _fields(words, bits):
    """All fields of 32-bit words [..., W] (int64): [..., W, 2 halves, 16/b]."""
    E = 16 // bits
    sh = torch.tensor([[16 * h + bits * e for e in range(E)] for h in range(2)], device=DEV)
    return (words[..., None, None] >> sh) & (2 ** bits - 1)


def _blocks64(s):
    """Values in 64 bits of every position of every block: K [n][Hkv][P][D],
    V the same, read by words instead of by bytes."""
    c = s["case"]
    D, bk, bv = c["head_dim"], c["bits_k"], c["bits_v"]
    n, Hkv, P = s["k_codes"].shape[:3]
    w = s["k_codes"].view(torch.int32).long().reshape(n, Hkv, P, 4, D * bk // 128)
    f = _fields(w, bk)  # [n][Hkv][P][slice c][word][half][e]: d = 8 * (word * E + e) + 2 c + half
    k = f.permute(0, 1, 2, 4, 6, 3, 5).reshape(n, Hkv, P, D)
    N, W = D * bv // 16, D * bv // 128
    piece = min(16, N)
    t = s["v_codes"].reshape(n, Hkv, P // 16, N // piece, 32, piece).transpose(3, 4)
    w = t.reshape(n, Hkv, P // 16, 8, 4, N).contiguous().view(torch.int32).long()
    f = _fields(w.reshape(n, Hkv, P // 16, 8, 4, 2, W), bv)
    # [..][tile][r][j][upper eight][word][half][e]: k = 8 * upper + 2 j + half, d = 8 * (word * E + e) + r
    v = f.permute(0, 1, 2, 5, 4, 7, 6, 8, 3).reshape(n, Hkv, P, D)
    kp, vp = s["k_params"].double(), s["v_params"].double()
    k = k.double().reshape(n, Hkv, P, -1, c["group"]) * kp[..., :1] + kp[..., 1:]
    v = v.double().reshape(n, Hkv, P, -1, _group_v(c)) * vp[..., :1] + vp[..., 1:]
    return k.reshape(n, Hkv, P, D), v.reshape(n, Hkv, P, D)


def _sylvester(D):
    i = np.arange(D)
    bits = i[:, None] & i[None, :]
    parity = np.zeros_like(bits)
    for k in range(8):
        parity ^= (bits >> k) & 1
    return torch.as_tensor(1.0 - 2.0 * parity, dtype=torch.float64, device=DEV)


def exact(case, seed):
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    D = case["head_dim"]
    if case["op"] == "append":
        # the codes are defined by binary32 steps, done here in numpy; the
        # values they stand for are taken in 64 bits
        out = {}
        params = {"k": s["k_params"].double(), "v": s["v_params"].double()}
        for name, bits, group in (("k", case["bits_k"], case["group"]),
                                  ("v", case["bits_v"], _group_v(case))):
            x = s[name].float().cpu().numpy()
            turn = name == "k" and case["rotate"]
            if turn:
                for h in [2 ** i for i in range(int(math.log2(D)))]:
                    lo = np.arange(D)[(np.arange(D) & h) == 0]
                    y = np.empty_like(x)
                    y[..., lo], y[..., lo + h] = x[..., lo] + x[..., lo + h], \
                        x[..., lo] - x[..., lo + h]
                    x = y
            x = x.reshape(x.shape[:2] + (-1, group))
            mn, mx = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
            scale = (mx - mn) / np.float32(2 ** bits - 1)
            with np.errstate(divide="ignore"):
                inv = np.float32(1.0) / scale
            ok = (scale > 0) & np.isfinite(scale) & np.isfinite(inv)
            code = np.where(ok, np.rint((x - mn) * np.where(ok, inv, np.float32(0))), 0)
            s16, z16 = scale.astype(np.float16), mn.astype(np.float16)
            val = code.astype(np.float64) * s16 + z16.astype(np.float64)
            val = torch.as_tensor(val.reshape(val.shape[:2] + (D,)), device=DEV)
            out[name] = val @ _sylvester(D) / D if turn else val
            par = np.concatenate((s16, z16), -1).astype(np.float64)
            params[name][s["block"], :, s["pos"]] = torch.as_tensor(par, device=DEV)
        return dict(k=out["k"], v=out["v"], k_params=params["k"], v_params=params["v"])
    k, v = _blocks64(s)
    P, gq = case["page"] or case["cap"], case["q_heads"] // case["kv_heads"]
    q = s["q"].double()
    if case["rotate"]:
        q = q @ _sylvester(D) / D
    old, new = _lens(case)
    cu, out = s["cu"].tolist(), torch.zeros_like(q)
    for b, (o, n) in enumerate(zip(old, new)):
        if n == o or n == 0:
            continue
        pages = s["table"][b, :(n + P - 1) // P].long() if case["page"] else \
            torch.tensor([b], device=DEV)
        kb = k[pages].transpose(0, 1).reshape(case["kv_heads"], -1, D)[:, :n]
        vb = v[pages].transpose(0, 1).reshape(case["kv_heads"], -1, D)[:, :n]
        seen = torch.arange(n, device=DEV)[None, :]
        for i in range(cu[b], cu[b + 1], 256):
            e = min(cu[b + 1], i + 256)
            lim = torch.arange(o + i - cu[b] + 1, o + e - cu[b] + 1, device=DEV)[:, None] \
                if case["causal"] else n
            x = torch.einsum("ihgd,htd->hgit", q[i:e].reshape(e - i, -1, gq, D), kb)
            x = (x / math.sqrt(D)).masked_fill(seen >= lim, -math.inf)
            out[i:e] = torch.einsum("hgit,htd->ihgd", x.softmax(-1), vb).reshape(e - i, -1, D)
    return out
