// Planning of a ragged step (kvq_plan_append): page allocation, block-table
// update, token offsets and the slot map, from the rows' lengths alone, in one
// launch and without a host round trip.
//
// Mathematics: prefix sums.  With have = ceil(old / P), want = ceil(new / P),
// a shrinking row returns table entries [want, have); a growing one needs
// want - have pages.  Row b's pages are the free pages of rank [upto_b -
// need_b, upto_b), upto the inclusive prefix sum of the needs and rank the
// exclusive prefix sum of (users == 0) over the pool; its 16-position tiles
// are the map entries [end_b - tiles_b, end_b) of the tiles' prefix sum.
// Every quantity is a whole number and every place follows from prefix sums,
// so the result does not depend on timing (the returns' atomic decrements
// commute).
//
// Bound: latency, one launch and up to three barriers, and for a large pool the
// read of its user counts (4 bytes a page).  One CTA's loads reach about 100
// GB/s, so a pool of more than kSmallPool pages is counted by a cluster of 8
// CTAs (the portable limit), each a contiguous part; the CTAs exchange their
// counts through distributed shared memory, and each repeats the rows' scans
// (a few microseconds for the largest batches, less than handing the results
// round).  The second sweep over the pool stops at the last page given out.
// Measured on B200, device time: 64 rows that grow by a token and are rolled
// back 14.1 us, two calls; 1000 rows with 134,000 pages and 12,000 map entries
// 36.8 us, two calls, the growing one about 23 us.
#include <cooperative_groups.h>

#include "common.cuh"
#include "internal.h"
#include "serve.h"

namespace kvq {
namespace {

namespace cg = cooperative_groups;

constexpr int kPlanThreads = 1024;
constexpr int kPlanCluster = 8;
// A cluster's barriers and start cost about as much as one CTA's sweep over
// this many user counts.
constexpr int kSmallPool = 8192;

// Sum of two counts, at most 2^31 - 1: rows may ask for more pages, tiles or
// tokens than 32 bits count.  Ascending prefix sums stay ascending, and a sum
// that was cut is more than any pool, map or tensor holds.
__device__ __forceinline__ int sat_add(int x, int y) {
  return static_cast<int>(min(static_cast<uint32_t>(x) + static_cast<uint32_t>(y), 0x7fffffffu));
}

// Inclusive prefix sum (saturating) over the CTA's threads of counts >= 0;
// *total: the CTA's sum.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, m);
    if (lane >= m) v = sat_add(v, u);
  }
  __syncthreads();  // the last scan's sums have been read
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  int s = warp_sums[lane];
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, s, m);
    if (lane >= m) s = sat_add(s, u);
  }
  *total = __shfl_sync(0xffffffffu, s, 31);
  const int before = __shfl_sync(0xffffffffu, s, max(warp - 1, 0));
  return sat_add(v, warp > 0 ? before : 0);
}

// First index in [0, n) whose (ascending) value exceeds x; n if none does.
__device__ __forceinline__ int first_above(const int* a, int n, int x) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] > x)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

// One row's request, checked: invalid lengths become a row that stays as it
// is (ok = false).
struct Row {
  int o, n;
  bool ok;
};

__device__ __forceinline__ Row load_row(const PlanArgs& a, int b) {
  Row r{a.old_lens[b], a.new_lens[b], true};  // (the planner's results of the call before, perhaps)
  if (r.o < 0 || r.n < 0 || r.o > a.capacity || r.n > a.capacity) {
    r.ok = false;
    r.n = r.o;
  }
  return r;
}

// Pages that a growing row takes.
__device__ __forceinline__ int pages_of(const PlanArgs& a, const Row& r) {
  const int P1 = (1 << a.page_shift) - 1;
  return ((r.n + P1) >> a.page_shift) - ((r.o + P1) >> a.page_shift);
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanArgs a) {
  extern __shared__ int smem[];
  int* s_upto = smem;               // [B] pages needed by the rows up to this one
  int* s_end = s_upto + a.batch;    // [B] tiles of the rows up to this one
  int* s_cu = s_end + a.batch;      // [B] tokens of the rows up to this one
  __shared__ int warp_sums[32];
  __shared__ int s_free;            // free pages of this CTA's part
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = cluster.block_rank(), parts = cluster.num_blocks();
  const int t = threadIdx.x;
  const int gtid = rank * kPlanThreads + t, gthreads = parts * kPlanThreads;
  const bool paged = a.table != nullptr;
  const int P1 = (1 << a.page_shift) - 1;
  pdl_wait();
  pdl_trigger();

  // ---- what the step does at all (every CTA finds the same): without growing
  // rows the pool is not counted, without shrinking ones nothing is returned,
  // and the barriers between go too
  bool shrinks = false, grows = false;
  for (int b = t; b < a.batch; b += kPlanThreads) {
    const Row r = load_row(a, b);
    shrinks |= r.n < r.o;
    grows |= r.n > r.o;
  }
  const bool returns = __syncthreads_or(shrinks) && paged;
  const bool takes = __syncthreads_or(grows) && paged;

  // ---- pages of shrinking rows go back to the pool: one warp a row
  if (returns) {
    for (int b = gtid / 32; b < a.batch; b += gthreads / 32) {
      const Row r = load_row(a, b);
      if (!r.ok || r.n >= r.o) continue;
      const int want = (r.n + P1) >> a.page_shift, have = (r.o + P1) >> a.page_shift;
      for (int j = want + (t & 31); j < have; j += 32) {
        int32_t* e = a.table + static_cast<size_t>(b) * a.pages_per_seq + j;
        const int page = *e;
        *e = -1;
        bool bad = page < 0 || page >= a.num_pages;
        if (!bad && atomicSub(a.users + page, 1) <= 0) {
          atomicAdd(a.users + page, 1);  // returned more often than it was taken
          bad = true;
        }
        if (bad) flag_error(a.err, KVQ_DEVERR_BAD_PAGE);
      }
    }
    if (takes) cluster.sync();
  }

  // ---- free pages of this CTA's part (whole vectors of 4)
  const int per = ((a.num_pages + parts - 1) / parts + 3) & ~3;
  const int lo = min(a.num_pages, rank * per), hi = min(a.num_pages, lo + per);
  const bool vec = (reinterpret_cast<uintptr_t>(a.users) & 15) == 0;
  auto load4 = [&](int i) {  // counts of pages i .. i + 3, 1 past the part
    int4 u = make_int4(1, 1, 1, 1);
    if (vec && i + 4 <= hi) {
      u = __ldcg(reinterpret_cast<const int4*>(a.users + i));
    } else {
      if (i < hi) u.x = __ldcg(a.users + i);
      if (i + 1 < hi) u.y = __ldcg(a.users + i + 1);
      if (i + 2 < hi) u.z = __ldcg(a.users + i + 2);
      if (i + 3 < hi) u.w = __ldcg(a.users + i + 3);
    }
    return u;
  };
  auto free4 = [](int4 u) { return (u.x == 0) + (u.y == 0) + (u.z == 0) + (u.w == 0); };
  int total = 0;
  if (takes) {
    int mine = 0;
#pragma unroll 4
    for (int i = lo + 4 * t; i < hi; i += 4 * kPlanThreads) mine += free4(load4(i));
    block_scan(mine, warp_sums, &total);
    if (t == 0) s_free = total;
  }

  // ---- rows: pages needed and tokens, summed up in row order
  int upto = 0, tokens = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kPlanThreads) {
    const int b = b0 + t;
    int need = 0, n_new = 0;
    if (b < a.batch) {
      const Row r = load_row(a, b);
      bool refused = !r.ok;
      if (refused && rank == 0)
        flag_error(a.err, r.o < 0 || a.new_lens[b] < 0 ? KVQ_DEVERR_BAD_POS
                                                               : KVQ_DEVERR_SEQ_LEN);
      if (r.n > r.o) {
        n_new = r.n - r.o;
        if (paged) {
          need = pages_of(a, r);
          if ((r.o & P1) != 0) {  // its last page takes tokens: it must be this row's alone
            const int page =
                a.table[static_cast<size_t>(b) * a.pages_per_seq + (r.o >> a.page_shift)];
            const bool inside = page >= 0 && page < a.num_pages;
            if (!inside || __ldcg(a.users + page) > 1) {
              refused = true;
              need = 0;
              if (rank == 0)
                flag_error(a.err, inside ? KVQ_DEVERR_NO_PAGE : KVQ_DEVERR_BAD_PAGE);
            }
          }
        }
      }
      s_end[b] = refused ? 1 : 0;  // (until the tiles' sums are written)
    }
    int sum;
    const int u = block_scan(need, warp_sums, &sum);
    if (b < a.batch) s_upto[b] = sat_add(upto, u);
    upto = sat_add(upto, sum);
    const int c = block_scan(n_new, warp_sums, &sum);
    if (b < a.batch) s_cu[b] = sat_add(tokens, c);
    tokens = sat_add(tokens, sum);
  }
  if (tokens > a.num_tokens && gtid == 0) flag_error(a.err, KVQ_DEVERR_CAPACITY);
  __syncthreads();

  // ---- free pages before this CTA's part, and in all
  int before = 0, all = 0;
  if (takes) {
    cluster.sync();
    for (int p = 0; p < parts; ++p) {
      const int f = *cluster.map_shared_rank(&s_free, p);
      if (p < rank) before += f;
      all += f;
    }
  }

  // ---- which rows are served; their tiles, summed up in row order
  int tiles_before = 0;
  int taken = 0;  // pages given out: the needs up to the last row that fits
  for (int b0 = 0; b0 < a.batch; b0 += kPlanThreads) {
    const int b = b0 + t;
    int tiles = 0;
    if (b < a.batch) {
      const Row r = load_row(a, b);
      bool refused = s_end[b] != 0;
      if (paged && !refused && r.n > r.o && pages_of(a, r) > 0) {
        if (s_upto[b] > all) {
          refused = true;
          if (rank == 0) flag_error(a.err, KVQ_DEVERR_NO_PAGE);
        } else {
          taken = max(taken, s_upto[b]);
        }
      }
      if (!refused && r.n > r.o) tiles = (r.n + 15) / 16 - r.o / 16;
      if (rank == 0) {
        a.lens[b] = refused ? r.o : r.n;
        if (b == 0) a.cu[0] = 0;
        a.cu[b + 1] = s_cu[b];
      }
    }
    int sum;
    const int e = block_scan(tiles, warp_sums, &sum);  // (every s_end of this pass was read)
    if (b < a.batch) s_end[b] = sat_add(tiles_before, e);
    tiles_before = sat_add(tiles_before, sum);
  }
  taken = __reduce_max_sync(0xffffffffu, taken);
  __syncthreads();
  if ((t & 31) == 0) warp_sums[t >> 5] = taken;
  __syncthreads();
  taken = __reduce_max_sync(0xffffffffu, warp_sums[t & 31]);

  // ---- free pages to rows: the page of rank r goes to the row whose needs
  // first reach past r
  if (takes) {
    for (int i0 = lo; i0 < hi && before < taken; i0 += 4 * kPlanThreads) {
      const int i = i0 + 4 * t;
      const int4 u = load4(i);
      int sum;
      const int mine = free4(u);
      int r = before + block_scan(mine, warp_sums, &sum) - mine;
      const int us[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if (us[x] != 0) continue;
        if (r < taken) {
          const int b = first_above(s_upto, a.batch, r);
          const int first = b > 0 ? s_upto[b - 1] : 0;
          const int have = (a.old_lens[b] + P1) >> a.page_shift;
          a.table[static_cast<size_t>(b) * a.pages_per_seq + have + (r - first)] = i + x;
          a.users[i + x] = 1;
        }
        ++r;
      }
      before += sum;
    }
    cluster.sync();  // the table is complete
  }

  // ---- the slot map: one entry per 16-position tile that takes tokens
  for (int e = gtid; e < a.num_entries; e += gthreads) {
    int4 m = make_int4(0, 0, 0, 0);
    const int b = first_above(s_end, a.batch, e);
    if (b < a.batch) {
      const Row r = load_row(a, b);
      const int tile = r.o / 16 + (e - (b > 0 ? s_end[b - 1] : 0));
      const int first = max(16 * tile, r.o), last = min(16 * tile + 16, r.n);
      const int token = sat_add(b > 0 ? s_cu[b - 1] : 0, first - r.o);
      int block = b;
      bool ok = true;
      if (paged) {
        block = __ldcg(a.table + static_cast<size_t>(b) * a.pages_per_seq +
                       ((16 * tile) >> a.page_shift));
        ok = block >= 0 && block < a.num_pages;
        if (!ok) flag_error(a.err, KVQ_DEVERR_BAD_PAGE);
      }
      const int count = min(last - first, a.num_tokens - token);
      if (ok && count > 0) m = make_int4(block, paged ? first & P1 : first, token, count);
    }
    a.map[e] = m;
  }
}

}  // namespace

cudaError_t launch_plan(const PlanArgs& a, cudaStream_t stream) {
  const size_t smem = sizeof(int) * 3 * static_cast<size_t>(a.batch);
  if (smem > 48 * 1024) {
    // The limit is one of the function and the device, whatever thread sets it:
    // always that of the largest batch, so that no call lowers another's
    // between its set and its launch.  (Once per call: it costs less than
    // keeping track of the devices.)
    const cudaError_t e =
        cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(sizeof(int)) * 3 * kPlanRows);
    if (e != cudaSuccess) return e;
  }
  const int parts = a.num_pages > kSmallPool ? kPlanCluster : 1;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = parts;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(parts);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, plan_kernel, a);
}

}  // namespace kvq
