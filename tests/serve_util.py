"""Plain references of the ragged serving step (64 bits, no kernel of the
library's attention) and input makers, shared by its GPU tests."""
import numpy as np
import torch

import kv_cache_mixed_kvq_b200 as kvq

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def plan_reference(old, new, table, users, P, capacity, batch):
    """(lens, cu, map entries, table, users, refused rows) of one planning call."""
    table, users = [list(r) for r in table], list(users)
    lens, cu, entries, refused = list(old), [0], [], set()
    pages = lambda n: (n + P - 1) // P  # noqa: E731
    bad = {b for b in range(batch) if not (0 <= old[b] <= capacity and 0 <= new[b] <= capacity)}
    for b in range(batch):
        if b not in bad and new[b] < old[b]:
            for j in range(pages(new[b]), pages(old[b])):
                users[table[b][j]] -= 1
                table[b][j] = -1
    free = [p for p, u in enumerate(users) if u == 0]
    want = 0
    taken = 0
    shared = {b for b in range(batch) if b not in bad and new[b] > old[b] and old[b] % P
              and users[table[b][old[b] // P]] > 1}
    for b in range(batch):
        n = 0 if b in bad else max(0, new[b] - old[b])
        cu.append(cu[-1] + n)
        if b in bad or b in shared:
            refused.add(b)
            continue
        need = max(0, pages(new[b]) - pages(old[b]))
        want += need
        if need and want > len(free):
            refused.add(b)
            continue
        for j in range(pages(old[b]), pages(old[b]) + need):
            table[b][j] = free[taken]
            users[free[taken]] = 1
            taken += 1
        lens[b] = new[b]
    for b in range(batch):
        p = old[b]
        while b not in refused and p < new[b]:
            e = min(new[b], p // 16 * 16 + 16)
            entries.append([table[b][p // P], p % P, cu[b] + p - old[b], e - p])
            p = e
    return lens, cu, entries, table, users, refused


def random_tables(rng, lens, P, cap, spare):
    """Scattered block tables for the rows' lengths, and the user counts."""
    have = [(n + P - 1) // P for n in lens]
    pool = max(1, sum(have) + spare)
    order = rng.permutation(pool)
    table = np.full((len(lens), cap // P), -1, np.int32)
    users = np.zeros(pool, np.int32)
    at = 0
    for b, h in enumerate(have):
        table[b, :h] = order[at:at + h]
        at += h
    users[order[:at]] = 1
    return table, users


def make_cache(B, Hkv, D, cap, bk, bv, G, gv=0, rotate=False, P=0, spare=0, seed=0, want=None):
    """A cache, its user counts, and (paged) tables with nothing cached yet."""
    if not P:
        return kvq.KVCache.allocate(B, Hkv, D, cap, bk, bv, G, group_v=gv, rotate_keys=rotate), None
    pool = sum((n + P - 1) // P for n in want) + spare
    table = torch.full((B, cap // P), -1, dtype=torch.int32)
    users = torch.zeros(max(1, pool), dtype=torch.int32, device="cuda")
    return kvq.KVCache.allocate(B, Hkv, D, cap, bk, bv, G, group_v=gv, rotate_keys=rotate,
                                page_size=P, num_pages=max(1, pool), block_table=table), users


def tokens(T, H, D, dtype, seed, spread=1.0, centre=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, D, generator=g) * spread + centre * torch.randn(1, H, D, generator=g)
    return x.to(DT[dtype]).cuda()


def fill(cache, users, lens, seed, dtype="bf16", centre=0.0):
    """Appends random tokens up to `lens` (planned from empty); returns the
    cached values (binary32 K, V [total][Hkv][D], K in its own basis) and cu."""
    B, total = cache.batch, int(sum(lens))
    out, cu, slots = kvq.kvq_plan_append(cache, i32([0] * B), i32(lens), total, users)
    k = tokens(total, cache.kv_heads, cache.head_dim, dtype, seed, centre=centre)
    v = tokens(total, cache.kv_heads, cache.head_dim, dtype, seed + 1)
    kvq.kvq_quantize_append_ragged(cache, k, v, slots)
    kd, vd = kvq.kvq_dequantize_ragged(cache, slots, total, torch.float32)
    assert kvq.kvq_device_error_flags() == 0
    return kd, vd, cu.tolist()


# Half a step of the number types, relative.
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def attention_reference(q, kd, vd, cu_kv, cu_q, lens, causal, scale, out_dtype, rot=False):
    """(o, tolerance) in 64 bits, both [T][Hq][D].

    Tolerance, for a kernel that takes binary16 operands and binary32 sums.
    With a query of 16-bit type exact, of binary32 to e_q = 2^-22 (two
    halves), of a rotated cache, where it is a sum H q / D, rounded like one
    (bf16 once, 2^-11; others in two halves; the products are then those of
    the rotated vectors); keys and values rounded once to binary16, e_k = e_v = 2^-11, for
    bf16 queries, held in two halves (2^-22) otherwise; weights e_p = 2^-11,
    2^-22 for binary32.  Roundings are independent and bounded, so by
    Hoeffding's inequality a sum of them stays within z times the root of the
    sum of squared bounds but with probability 2 exp(-z^2/2) (z = 7: 5e-11):
      d s_t <= z sqrt(sum_d (q_d k_td)^2) scale (e_q + e_k) = z a_t,
      d o   <= z sqrt(sum_t p_t^2 ((v_t - o)^2 a_t^2 + v_t^2 (e_p^2 + e_v^2))).
    (With one visible position p = 1 whatever s is: the first term vanishes.)
    To these come, without a sign to count on, binary32 sums: a score's D/16
    chained products of up to 3 pieces, each off by at most 2^-23 of the sum
    of magnitudes A_t, and the exponential's argument and value (2^-22):
      d s_t <= (3 D/16 + 4) 2^-23 A_t + 2^-21,
    and the n/16 chained products of the output, again taken as independent
    (z sqrt(n/16 + 4) 2^-23 sum_t p_t |v_t|); the rescalings and the quotient
    (8 * 2^-24 |o|), and the output's rounding, half a step of its type (or
    of the smallest binary16, 2^-25)."""
    T, Hq, D = q.shape
    gq = Hq // kd.shape[1]
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    kind = q.dtype
    e_q = 2.0 ** -22 if kind == torch.float32 else 0.0
    if rot:
        e_q = 2.0 ** -11 if kind == torch.bfloat16 else 2.0 ** -22
        H = torch.ones(1, 1, dtype=torch.float64, device=q.device)
        while H.shape[0] < D:
            H = torch.cat([torch.cat([H, H], 1), torch.cat([H, -H], 1)], 0)
    e_kv = 2.0 ** -11 if kind == torch.bfloat16 else 2.0 ** -22
    e_p = 2.0 ** -22 if kind == torch.float32 else 2.0 ** -11
    z = 7.0
    scale = scale if scale > 0 else D ** -0.5
    for b in range(len(lens)):
        n, L = cu_q[b + 1] - cu_q[b], lens[b]
        if n == 0:
            continue
        k = kd[cu_kv[b]:cu_kv[b] + L].double().repeat_interleave(gq, 1)
        v = vd[cu_kv[b]:cu_kv[b] + L].double().repeat_interleave(gq, 1)
        if rot:
            k = k @ H
        for i0 in range(0, n, 128):
            sl = slice(cu_q[b] + i0, cu_q[b] + min(n, i0 + 128))
            x = q[sl].double()
            if rot:
                x = x @ H / D
            i = torch.arange(i0, min(n, i0 + 128), device=q.device)
            seen = (L - n + i + 1 if causal else torch.full_like(i, L)).clamp(0, L)
            if L == 0:
                continue
            s = torch.einsum("ihd,thd->hit", x, k) * scale
            A = torch.einsum("ihd,thd->hit", x.abs(), k.abs()) * scale
            a = torch.einsum("ihd,thd->hit", x ** 2, k ** 2).sqrt() * scale * (e_q + e_kv)
            mask = torch.arange(L, device=q.device)[None, :] >= seen[:, None]
            p = torch.softmax(s.masked_fill(mask, float("-inf")), -1).nan_to_num(0.0)
            o = torch.einsum("hit,thd->ihd", p, v)
            w = (p * a) ** 2
            var = torch.einsum("hit,thd->ihd", w, v ** 2) \
                - 2 * o * torch.einsum("hit,thd->ihd", w, v) \
                + o ** 2 * w.sum(-1).T[..., None]
            var = var.clamp(min=0) + torch.einsum("hit,thd->ihd", p ** 2, v ** 2) * \
                (e_p ** 2 + e_kv ** 2)
            ds = (3 * D / 16 + 4) * 2.0 ** -23 * A + 2.0 ** -21
            pv = torch.einsum("hit,thd->ihd", p, v.abs())
            flat = torch.einsum("hit,thd->ihd", p * ds, v.abs()) + \
                o.abs() * (p * ds).sum(-1).T[..., None]
            flat += z * (L / 16 + 4) ** 0.5 * 2.0 ** -23 * pv + 8 * 2.0 ** -24 * o.abs()
            t = z * var.sqrt() + flat
            half = HALF[out_dtype] * (o.abs() + t)
            if out_dtype == torch.float16:
                half = half.clamp(min=2.0 ** -25)
            out[sl], tol[sl] = o, t + half
    return out, tol


def assert_close(got, want, tol):
    err = (got.double() - want).abs()
    assert torch.isfinite(got.float()).all(), "non-finite output"
    bad = (err > tol).nonzero()
    if bad.numel():
        i = tuple(bad[0].tolist())
        raise AssertionError(f"{len(bad)} of {err.numel()} outputs off, first at {i}: got "
                             f"{got[i].item():.6g}, want {want[i].item():.6g}, "
                             f"tolerance {tol[i].item():.2e}")
