// Host side of the ragged serving step's entry points: argument checks and
// launches.  No allocation anywhere.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "host.h"
#include "serve.h"

namespace {

using namespace kvq;

BlockCache block_cache(const kvq_cache_desc* c) {
  BlockCache b;
  b.k_codes = c->k_codes;
  b.v_codes = c->v_codes;
  b.k_params = static_cast<uint32_t*>(c->k_params);
  b.v_params = static_cast<uint32_t*>(c->v_params);
  b.kv_heads = c->kv_heads;
  b.head_dim = c->head_dim;
  b.bits_k = c->bits_k;
  b.bits_v = c->bits_v;
  b.group = c->group;
  b.group_v = group_v_of(c);
  b.gshift_k = b.group == 32 ? 5 : b.group == 64 ? 6 : 7;
  b.gshift_v = b.group_v == 32 ? 5 : b.group_v == 64 ? 6 : 7;
  const bool paged = (c->flags & KVQ_FLAG_PAGED) != 0;
  b.blocks = paged ? c->num_pages : c->batch;
  b.block_tokens = paged ? c->page_size : c->capacity;
  b.rotate_keys = (c->flags & KVQ_FLAG_ROTATE_KEYS) != 0;
  return b;
}

// Whether tokens of `heads` heads may lie `stride` elements apart: no overlap,
// and every token on a 16-byte boundary.
bool valid_stride(int64_t stride, int heads, int D, int dtype) {
  return stride >= static_cast<int64_t>(heads) * D && stride % (dtype == KVQ_F32 ? 4 : 8) == 0;
}

int ragged_impl(const kvq_cache_desc* cache, const void* k, int64_t k_stride, const void* v,
                int64_t v_stride, int32_t dtype, int32_t num_tokens, const int32_t* slot_map,
                int32_t num_entries, bool append, kvq_stream_t stream) {
  int st = check_cache(cache);
  if (st != KVQ_OK) return st;
  if (!valid_dtype(dtype) || num_tokens < 0 || num_entries < 0) return KVQ_ERR_INVALID_ARG;
  if (num_tokens == 0 || num_entries == 0) return KVQ_OK;
  if (!k || !v || !slot_map || !aligned(k, 16) || !aligned(v, 16) || !aligned(slot_map, 16) ||
      !valid_stride(k_stride, cache->kv_heads, cache->head_dim, dtype) ||
      !valid_stride(v_stride, cache->kv_heads, cache->head_dim, dtype))
    return KVQ_ERR_INVALID_ARG;
  RaggedArgs a;
  a.c = block_cache(cache);
  a.k = k;
  a.v = v;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.dtype = dtype;
  a.num_tokens = num_tokens;
  a.num_entries = num_entries;
  a.map = reinterpret_cast<const int4*>(slot_map);
  st = error_word(&a.err);
  if (st != KVQ_OK) return st;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return to_status(append ? launch_append_ragged(a, s) : launch_dequantize_ragged(a, s));
}

// Positions are counted in 32 bits, rounded up to tiles and pages.
constexpr int kMaxLength = 1 << 30;

int check_chunk(const kvq_cache_desc* c, int Hq, int num_tokens, int max_q_len, int max_seq_len) {
  const int st = check_cache(c);
  if (st != KVQ_OK) return st;
  if (Hq < 1 || Hq % c->kv_heads != 0 || num_tokens < 0 || max_q_len < 0 || max_seq_len < 0)
    return KVQ_ERR_INVALID_ARG;
  if (c->batch > kChunkRows || std::min(max_seq_len, c->capacity) > kMaxLength)
    return KVQ_ERR_UNSUPPORTED;
  // the (token, query head) rows are counted in 32 bits
  if (static_cast<long long>(num_tokens) * Hq > 0x7fffffffll / 2) return KVQ_ERR_UNSUPPORTED;
  // and so are a kv head's steps: units of at least 128 rows by tiles
  const long long units =
      static_cast<long long>(num_tokens) * (Hq / c->kv_heads) / 128 + std::min(c->batch, num_tokens);
  const long long tiles = std::min(max_seq_len, c->capacity) / 64 + 1 + kUnitCost;
  if (units * tiles > 0x7fffffffll / 2) return KVQ_ERR_UNSUPPORTED;
  return KVQ_OK;
}

// Binary16 pieces of the operands (see chunk.cuh).  A rotated binary16 query
// is a sum, no longer exact in one piece.
int pieces_of(const kvq_cache_desc* c, int q_dtype) {
  if (q_dtype == KVQ_BF16) return 1;
  return q_dtype == KVQ_F32 || (c->flags & KVQ_FLAG_ROTATE_KEYS) ? 3 : 2;
}

struct ChunkPlan {
  int grid, max_units, part_rows;
  bool whole_units;
  size_t ml_offset, o_offset, bytes;  // workspace: headers, (m, l), o
};

// Steps up to which a unit is not worth dividing: the set-up of a CTA and the
// joining of its partial results cost more than the steps.
constexpr int kWholeSteps = 2;
constexpr int kMinShare = kWholeSteps + kUnitCost;

// Division of work, from the host's bounds alone (the lengths are on the
// device): one CTA per SM, fewer when there cannot be that much work.  Units
// of at most kWholeSteps steps stay whole, which saves the joining launch.
int chunk_plan(const kvq_cache_desc* c, int Hq, int num_tokens, int max_q_len, int max_seq_len,
               int pieces, ChunkPlan* p) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return KVQ_ERR_CUDA;
  const int gq = Hq / c->kv_heads, unit = unit_rows(pieces);
  const int q_len = std::min(max_q_len, num_tokens);
  const long long rows = static_cast<long long>(q_len) * gq;
  const long long units =
      (static_cast<long long>(num_tokens) * gq / unit + std::min(c->batch, num_tokens)) *
      c->kv_heads;
  const int len = std::min(max_seq_len, c->capacity);
  const int tile = tile_tokens(pieces, c->head_dim, c->bits_k + c->bits_v);
  const long long tiles = (len + tile - 1) / tile;
  const long long steps = std::max(1ll, rows > 128 && unit > 128 ? tiles : (tiles + 1) / 2);
  p->whole_units = steps <= kWholeSteps;
  p->max_units = static_cast<int>((rows + unit - 1) / unit);
  p->grid = static_cast<int>(std::min<long long>(
      sms, p->whole_units ? units : (units * (steps + kUnitCost) + kMinShare - 1) / kMinShare));
  p->grid = std::max(1, p->grid);
  p->part_rows = static_cast<int>(std::min<long long>(unit, std::max(1ll, rows)));
  const size_t places = static_cast<size_t>(p->grid) * 2;
  p->ml_offset = places * 32;
  p->o_offset = (p->ml_offset + places * p->part_rows * 8 + 15) / 16 * 16;
  p->bytes = p->whole_units ? 0 : p->o_offset + places * p->part_rows * c->head_dim * 4;
  return KVQ_OK;
}

// As many tokens as batch rows, one a row at most: a decode step, some of its
// rows idle perhaps, which is the decode kernel's case for 16-bit types.
bool is_decode(const kvq_cache_desc* c, int num_tokens, int max_q_len, int max_seq_len) {
  return max_q_len == 1 && num_tokens == c->batch && max_seq_len > 0;
}

// Workspace of a call, whatever its element types (arguments checked).
size_t chunk_workspace(const kvq_cache_desc* c, int Hq, int num_tokens, int max_q_len,
                       int max_seq_len) {
  size_t need = 0;
  for (int pieces = 1; pieces <= 3; ++pieces) {
    ChunkPlan p;
    if (chunk_plan(c, Hq, num_tokens, max_q_len, max_seq_len, pieces, &p) != KVQ_OK) return 0;
    need = std::max(need, p.bytes);
  }
  if (is_decode(c, num_tokens, max_q_len, max_seq_len))
    need = std::max(need, kvq_decode_workspace_bytes(c, Hq, max_seq_len));
  return need;
}

}  // namespace

extern "C" {

int32_t kvq_slot_map_entries(int32_t batch, int32_t num_tokens) {
  if (batch < 0 || num_tokens < 0) return 0;
  return static_cast<int32_t>(
      std::min<int64_t>(num_tokens, num_tokens / 16 + 2 * static_cast<int64_t>(batch)));
}

int kvq_plan_append(const kvq_cache_desc* cache, const int32_t* old_lens,
                    const int32_t* new_lens, int32_t num_tokens, int32_t* page_users,
                    int32_t* lens, int32_t* cu_tokens, int32_t* slot_map, int32_t num_entries,
                    kvq_stream_t stream) {
  int st = check_cache(cache);
  if (st != KVQ_OK) return st;
  if (cache->batch > kPlanRows || cache->capacity > kMaxLength) return KVQ_ERR_UNSUPPORTED;
  const bool paged = (cache->flags & KVQ_FLAG_PAGED) != 0;
  if (!old_lens || !new_lens || !lens || !cu_tokens || !aligned(old_lens, 4) ||
      !aligned(new_lens, 4) || !aligned(lens, 4) || !aligned(cu_tokens, 4) || num_tokens < 0 ||
      lens == old_lens || lens == new_lens ||  // (read again after lens is written)
      num_entries < kvq_slot_map_entries(cache->batch, num_tokens) ||
      (num_entries > 0 && (!slot_map || !aligned(slot_map, 16))) ||
      paged != (page_users != nullptr) || !aligned(page_users, 4))
    return KVQ_ERR_INVALID_ARG;
  PlanArgs a;
  a.old_lens = old_lens;
  a.new_lens = new_lens;
  a.batch = cache->batch;
  a.capacity = cache->capacity;
  a.num_tokens = num_tokens;
  a.num_entries = num_entries;
  a.users = page_users;
  const int32_t* table;
  page_args(cache, &table, &a.page_shift, &a.pages_per_seq, &a.num_pages);
  a.table = const_cast<int32_t*>(table);  // the caller's table: this call updates it
  a.lens = lens;
  a.cu = cu_tokens;
  a.map = reinterpret_cast<int4*>(slot_map);
  st = error_word(&a.err);
  if (st != KVQ_OK) return st;
  return to_status(launch_plan(a, reinterpret_cast<cudaStream_t>(stream)));
}

int kvq_quantize_append_ragged(const kvq_cache_desc* cache, const void* k, int64_t k_stride,
                               const void* v, int64_t v_stride, int32_t in_dtype,
                               int32_t num_tokens, const int32_t* slot_map, int32_t num_entries,
                               kvq_stream_t stream) {
  return ragged_impl(cache, k, k_stride, v, v_stride, in_dtype, num_tokens, slot_map, num_entries,
                     true, stream);
}

int kvq_dequantize_ragged(const kvq_cache_desc* cache, const int32_t* slot_map,
                          int32_t num_entries, void* k_out, void* v_out, int32_t out_dtype,
                          int32_t num_tokens, kvq_stream_t stream) {
  const int64_t stride =
      cache ? static_cast<int64_t>(cache->kv_heads) * cache->head_dim : 0;  // packed outputs
  return ragged_impl(cache, k_out, stride, v_out, stride, out_dtype, num_tokens, slot_map,
                     num_entries, false, stream);
}

size_t kvq_chunk_workspace_bytes(const kvq_cache_desc* cache, int32_t num_q_heads,
                                 int32_t num_tokens, int32_t max_q_len, int32_t max_seq_len) {
  if (check_chunk(cache, num_q_heads, num_tokens, max_q_len, max_seq_len) != KVQ_OK) return 0;
  return chunk_workspace(cache, num_q_heads, num_tokens, max_q_len, max_seq_len);
}

int kvq_chunk_attention(const kvq_cache_desc* cache, const void* q, int64_t q_stride,
                        int32_t q_dtype, int32_t num_q_heads, int32_t num_tokens,
                        const int32_t* cu_tokens, const int32_t* seq_lens, int32_t max_q_len,
                        int32_t max_seq_len, int32_t causal, float sm_scale, void* out,
                        int32_t out_dtype, void* workspace, size_t workspace_bytes,
                        kvq_stream_t stream) {
  int st = check_chunk(cache, num_q_heads, num_tokens, max_q_len, max_seq_len);
  if (st != KVQ_OK) return st;
  if (!valid_dtype(q_dtype) || !valid_dtype(out_dtype) || !(sm_scale == sm_scale))
    return KVQ_ERR_INVALID_ARG;
  if (num_tokens == 0) return KVQ_OK;
  if (!q || !out || !cu_tokens || !seq_lens || !aligned(q, 16) || !aligned(out, 16) ||
      !aligned(cu_tokens, 4) || !aligned(seq_lens, 4) ||
      !valid_stride(q_stride, num_q_heads, cache->head_dim, q_dtype))
    return KVQ_ERR_INVALID_ARG;
  if (is_decode(cache, num_tokens, max_q_len, max_seq_len) && q_dtype != KVQ_F32 &&
      q_stride == static_cast<int64_t>(num_q_heads) * cache->head_dim)
    return decode_single_tokens(cache, q, q_dtype, num_q_heads, num_tokens, cu_tokens, seq_lens,
                                max_seq_len, sm_scale, out, out_dtype, workspace, workspace_bytes,
                                stream);
  const int pieces = pieces_of(cache, q_dtype);
  ChunkPlan p;
  st = chunk_plan(cache, num_q_heads, num_tokens, max_q_len, max_seq_len, pieces, &p);
  if (st != KVQ_OK) return st;
  if (p.bytes > 0 &&
      (!workspace || !aligned(workspace, 16) ||
       workspace_bytes < chunk_workspace(cache, num_q_heads, num_tokens, max_q_len, max_seq_len)))
    return KVQ_ERR_WORKSPACE;
  const float scale =
      sm_scale > 0.0f ? sm_scale : 1.0f / sqrtf(static_cast<float>(cache->head_dim));
  ChunkArgs a;
  a.c = block_cache(cache);
  int num_pages;
  page_args(cache, &a.table, &a.page_shift, &a.pages_per_seq, &num_pages);
  a.batch = cache->batch;
  a.capacity = cache->capacity;
  a.q = q;
  a.q_stride = q_stride;
  a.q_dtype = q_dtype;
  a.q_heads = num_q_heads;
  a.gq = num_q_heads / cache->kv_heads;
  a.num_tokens = num_tokens;
  a.cu = cu_tokens;
  a.seq_lens = seq_lens;
  a.max_q_len = max_q_len;
  a.max_seq_len = max_seq_len;
  a.causal = causal != 0;
  a.sm_scale_log2 = scale * 1.4426950408889634f;
  a.out = out;
  a.out_dtype = out_dtype;
  a.whole_units = p.whole_units;
  a.min_share = p.whole_units ? 1 : kMinShare;
  a.max_units = p.max_units;
  a.part_rows = p.part_rows;
  uint8_t* ws = p.bytes > 0 ? static_cast<uint8_t*>(workspace) : nullptr;
  a.ws_head = reinterpret_cast<int*>(ws);
  a.ws_ml = reinterpret_cast<float2*>(ws ? ws + p.ml_offset : nullptr);
  a.ws_o = reinterpret_cast<float*>(ws ? ws + p.o_offset : nullptr);
  st = error_word(&a.err);
  if (st != KVQ_OK) return st;
  unsigned long long limit;
  a.fault_stage = take_fault(&limit);
  a.wait_limit_ns = static_cast<uint32_t>(limit);  // (a second at most)
  return to_status(launch_chunk(a, pieces, p.grid, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
