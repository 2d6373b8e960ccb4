// Attention of a chunk of new tokens over the packed cache
// (kvq_chunk_attention), on the Blackwell tensor cores.
//
//   s_it = scale q_i . k^_t,  p_it = exp(s_it - m_i),  o_i = sum_t p_it v^_t / sum_t p_it
// in one pass over the positions t with a running reference m_i of the
// exponents: m_i follows the running maximum, but o_i and l_i = sum_t p_it are
// rescaled (by exp(m_i - m_i')) only when the maximum has grown by more than a
// factor 2^kThreshold, since any reference cancels in the quotient.  The query
// heads of one kv head share its keys, so a row of a tile is a (token, head)
// pair: row r of batch row b is its new token r / gq, head r mod gq of the kv
// head.
//
// Products: S = Q K^T and O += P V by tcgen05.mma (kind::f16, binary32
// accumulators in tensor memory), 128 rows x NT positions x D.  Operands are
// binary16, keys and values unpacked to it in the kernel.  How many binary16
// pieces hold an operand follows from the query's type (PIECES):
//   1  bf16: a query row, scaled by a power of two, is exact in binary16; keys,
//      values and weights are rounded once, 2^-11, an eighth of the output's
//      2^-8;
//   2  f16: query exact, keys and values in two pieces (hi + lo, 2^-22): a
//      score's error is the keys' relative error times the sum of magnitudes,
//      which one piece would make several times the output's 2^-11;
//   3  f32: query, keys, weights and values in two pieces, products hi hi +
//      hi lo + lo hi, 2^-22 in all.
// Softmax statistics, sums and outputs are binary32.
//
// Roles (28 warps, one CTA per SM):
//   warps 0-15  softmax: two slots of eight warps; two threads a row of a slot
//   warps 16-23 unpacking, those of SM quarters 0 and 1 the keys: packed codes
//               from the ring to a K tile (binary16, 128-byte swizzle), those
//               of quarters 2 and 3 the values, to a V tile (rows are
//               elements: K-major along the positions, which is the order of
//               the packed V tiles).  A quarter that holds the code of one of
//               them alone was 1 to 6 % faster.
//   warp 24     issues the MMAs
//   warp 25     walks the work list and publishes each piece of work
//   warps 26-27 copy packed codes and parameters, 32 positions at a time, into
//               the ring (cp.async: four bulk copies a block, issued by one
//               lane, took 900 cycles)
// In a wide unit (more than 128 rows) the slots are its two halves and share
// each K and V tile; in a narrow one they take alternate tiles of the same
// rows and are merged at the end, so that one slot's softmax runs while the
// other's products do.
//
// Work: units of up to UNIT rows of one kv head, each a number of steps (one
// tile for both slots, or one tile a slot).  All units' steps are laid end to
// end and every CTA takes an equal share, so that ragged lengths, few rows
// with long contexts and more units than SMs all fill the card.  A unit cut by
// a share's border leaves partial results (o, m, l) that combine_kernel joins;
// whole units write their output directly.  The division depends on the
// lengths and the grid alone, so results do not depend on timing.
//
// Bound: the issue of instructions and their latency, not a pipe.  A step of a
// wide unit (256 rows x 128 positions, D = 128, 16.8 MFLOP) takes about 5000
// cycles; of these the tensor pipe is busy for 2000 (its products alone, as
// issued here, take 2800: 102 cycles per 128 x 128 x 16 product with both
// operands in shared memory, 73 with the weights in tensor memory), the
// exponentials 2000, and 12,300 warp instructions are issued (63 % of issue
// slots).  Between two products of a slot lies its softmax, whose chain
// (scores, maxima, exchange, weights) is what the other slot's products
// hide.  Measured on B200: 2048 queries of 32 heads (8 kv heads, K4V2) at
// position 24576, 0.97-1.02 ms = 0.84-0.88 PFLOP/s (half of the measured bf16
// peak of 1.66); ragged prefill of 4 x 2000-4000 tokens, 0.488 ms = 0.60
// PFLOP/s.  Narrow units are bound by the same chain with few valid rows: 16
// rows x 4 tokens x 4256 positions on average, 88 us (0.72 TB/s of cache bytes).
// What was measured and not kept, in us for these three cases where the kept
// form of its time took 1010, 558 and 107: tiles of 64 positions with the next
// tile's scores ahead of the softmax (1124, 791, 135), weights held in registers
// while the maximum is found (1421, 917, 167: unrolled code leaves the
// instruction caches).
#pragma once

#include "common.cuh"
#include "internal.h"
#include "serve.h"
#include "tc.cuh"

namespace kvq {
namespace chunk {

constexpr int kThreads = 28 * 32;
constexpr int kWarpUnpack = 16, kWarpMma = 24, kWarpList = 25, kWarpCopy = 26;
constexpr int kCopiers = 2;       // warps that copy, block by block in turn
// Registers a thread at launch, and of each warpgroup after the split: 512 x 80
// + 256 x 64 + 128 x 56 <= 896 x 72.  (Seven warps share an SM quarter's 16384
// registers, hence 72: what 65 to 72 allocate, in eights.)
constexpr int kRegsLaunch = 72, kRegsSoftmax = 80, kRegsUnpack = 64, kRegsIssue = 56;
static_assert(512 * kRegsSoftmax + 256 * kRegsUnpack + 128 * kRegsIssue <= kThreads * kRegsLaunch,
              "more registers than the launch has would never be granted");
constexpr int kRing = 16;         // ring blocks at most
constexpr int kBlock = 32;        // positions of a ring block
constexpr int kSmemMax = 232448;   // shared memory a CTA may have (227 KB)
constexpr int kHeader = 7 * 1024;  // barriers, pieces, exchanged maxima and sums

template <int D_, int PIECES_, int NT_>
struct Cfg {
  static constexpr int D = D_, PIECES = PIECES_;
  static constexpr int NT = NT_;                     // positions of a tile
  static constexpr int KP = PIECES == 1 ? 1 : 2;     // pieces of a key or value
  static constexpr int UNIT = unit_rows(PIECES);     // rows of a unit
  static constexpr int BLOCKS = NT / kBlock;
  static constexpr int PARTS = 4 / BLOCKS;           // warps that share a ring block
  static constexpr int QTILE = 128 * D * 2;          // bytes of one Q region
  static constexpr int KPIECE = NT * D * 2;
  static constexpr int STAGE = KPIECE * KP;          // bytes of a K or V tile
  static constexpr int SMEM_K = 2 * QTILE;
  static constexpr int SMEM_V = SMEM_K + 2 * STAGE;
  static constexpr int SMEM_RING = SMEM_V + 2 * STAGE;
  // tensor memory columns: S (P in its place) and O of each slot
  static constexpr int S_COL = 128, O_COL = 128, O_BASE = 256;
  // weights are 2^(x - m + kOffset): their smallest binary16 values lie that
  // much below the largest ones, which stay below 2^(kOffset + kThreshold)
  static constexpr float kOffset = PIECES == 3 ? 11.0f : 7.0f;
  static constexpr float kThreshold = PIECES == 3 ? 4.0f : 8.0f;
};

// One piece of work: steps [j0, j1) of a unit.
struct Piece {
  int valid, h, start, n, len;  // batch row: first packed token, tokens, length
  int row0, rows, wide;         // unit's first row, number of rows
  int lim;                      // positions that its last row sees
  int t0, t1;                   // tiles the piece needs, [t0, t1)
  int nt0;                      // wide: tiles of slot 0
  int j0, j1;
  int begin, end;               // whether it holds the unit's first and last step
  int b;
  int pad[15];
};
static_assert(sizeof(Piece) == 128, "");

struct Shared {
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t s_full[2], p_full[2];
  uint64_t q_full, m_full, m_free;
  uint64_t drained;  // the products in flight when a wait ran out
  uint32_t tokens[2];  // of all usable rows: sums of the low 16 bits and of the others
  uint64_t x_full[2][4];  // [slot][quarter of the rows]: the two halves' maxima
  uint64_t d_full[2], d_empty[2];
  uint64_t ring_full[kRing], ring_empty[kRing];
  uint32_t tmem;
  int abort;
  int total;  // steps of one kv head's units
  int pad;
  Piece piece[2];
  float2 stat[128];  // narrow merge: slot 1's (m, l)
  float unscale[2][128];  // of each slot's query rows
  float top[2][2][2][128];  // [slot][turn][half of the columns]: maxima or sums
};
static_assert(sizeof(Shared) <= kHeader, "header");

struct Waiter {
  int* abort;
  uint32_t limit_ns;
  // Bounded wait of a warp: false if the phase did not complete within the
  // limit, or if another wait of this CTA gave up (the kernel's end flags it).
  // The loop is short: it is part of every role's code.
  __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const {
    bool ok = mbar_try_wait(bar, parity);
    if (!ok) {
      const uint32_t t0 = timer();
      while (!(ok = mbar_try_wait(bar, parity))) {
        if (timer() - t0 > limit_ns)
          *reinterpret_cast<volatile int*>(abort) = 1;
        if (*reinterpret_cast<volatile int*>(abort) != 0) break;
      }
    }
    return __all_sync(0xffffffffu, ok) != 0;
  }
  static __device__ __forceinline__ uint32_t timer() {  // nanoseconds, mod 2^32
    uint32_t t;
    asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
    return t;
  }
};

// ------------------------------------------------------------------- work
// Tokens of batch row b; n = 0 if its offsets are not usable.
struct RowInfo {
  int start, n, len;
  bool bad, longer;
};

__device__ __forceinline__ RowInfo row_info(const ChunkArgs& a, int b) {
  RowInfo r;
  // (coherent loads, as everywhere that the planner may just have written: the
  // launch may have begun before it ended)
  r.start = a.cu[b];
  const int end = a.cu[b + 1];
  r.bad = r.start < 0 || end < r.start || end - r.start > a.max_q_len || end > a.num_tokens;
  r.n = r.bad ? 0 : end - r.start;
  const int lim = min(a.max_seq_len, a.capacity);
  const int len = a.seq_lens[b];
  r.longer = len > lim;
  r.len = max(0, min(len, lim));
  return r;
}

// Positions that unit row r (of batch row tokens n, length len) sees.
__device__ __forceinline__ int limit_of(const ChunkArgs& a, int n, int len, int r) {
  return a.causal ? max(0, min(len, len - n + r / a.gq + 1)) : len;
}

struct Unit {
  int row0, rows, wide, lim, nt, nt0, steps;
};

template <class C>
__device__ __forceinline__ Unit unit_of(const ChunkArgs& a, int n, int len, int m) {
  Unit u;
  u.row0 = m * C::UNIT;
  u.rows = min(C::UNIT, n * a.gq - u.row0);
  u.wide = u.rows > 128;
  u.lim = limit_of(a, n, len, u.row0 + u.rows - 1);
  u.nt = (u.lim + C::NT - 1) / C::NT;
  u.nt0 = u.wide ? (limit_of(a, n, len, u.row0 + 127) + C::NT - 1) / C::NT : 0;
  u.steps = max(1, u.wide ? u.nt : (u.nt + 1) / 2);
  return u;
}

// What a unit counts in the division of work: its steps and what its queries
// and output take.
template <class C>
__device__ __forceinline__ int unit_cost(const ChunkArgs& a, int n, int len, int m) {
  return a.whole_units ? 1 : unit_of<C>(a, n, len, m).steps + kUnitCost;
}

__device__ __forceinline__ int warp_sum(int v) {
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

__device__ __forceinline__ int warp_scan(int v, int lane) {  // inclusive
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, m);
    if (lane >= m) v += u;
  }
  return v;
}

// Whether the usable rows have more tokens than there are (see scan_rows).
__device__ __forceinline__ bool overlapping(const ChunkArgs& a, const Shared* sh) {
  return (static_cast<unsigned long long>(sh->tokens[1]) << 16) + sh->tokens[0] >
         static_cast<unsigned long long>(a.num_tokens);
}

// Inclusive prefix sums of the rows' costs into pref[0 .. batch) (all warps;
// ends with a CTA barrier); the errors of unusable rows are flagged once.
// Offsets that do not ascend can leave rows that overlap, with more tokens in
// all than there are and more work than 32 bits count: then there is none.
template <class C>
__device__ __forceinline__ void scan_rows(const ChunkArgs& a, int* pref, Shared* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool reports = blockIdx.x == 0;
  uint32_t tokens_lo = 0, tokens_hi = 0;
  if (a.max_units > 8) {  // long chunks: a warp per row
    for (int b = warp; b < a.batch; b += kThreads / 32) {
      const RowInfo r = row_info(a, b);
      const int mt = (r.n * a.gq + C::UNIT - 1) / C::UNIT;
      int c = 0;
      for (int m = lane; m < mt; m += 32) c += unit_cost<C>(a, r.n, r.len, m);
      c = warp_sum(c);
      if (lane == 0) {
        tokens_lo += r.n & 0xffff;
        tokens_hi += r.n >> 16;
        pref[b] = c;
        if (reports && r.bad) flag_error(a.err, KVQ_DEVERR_BAD_POS);
        if (reports && r.longer) flag_error(a.err, KVQ_DEVERR_SEQ_LEN);
      }
    }
  } else {
    for (int b = threadIdx.x; b < a.batch; b += kThreads) {
      const RowInfo r = row_info(a, b);
      const int mt = (r.n * a.gq + C::UNIT - 1) / C::UNIT;
      int c = 0;
      for (int m = 0; m < mt; ++m) c += unit_cost<C>(a, r.n, r.len, m);
      tokens_lo += r.n & 0xffff;
      tokens_hi += r.n >> 16;
      pref[b] = c;
      if (reports && r.bad) flag_error(a.err, KVQ_DEVERR_BAD_POS);
      if (reports && r.longer) flag_error(a.err, KVQ_DEVERR_SEQ_LEN);
    }
  }
  __syncthreads();
  tokens_lo = __reduce_add_sync(0xffffffffu, tokens_lo);
  tokens_hi = __reduce_add_sync(0xffffffffu, tokens_hi);
  if (lane == 0 && (tokens_lo | tokens_hi) != 0) {
    atomicAdd(&sh->tokens[0], tokens_lo);
    atomicAdd(&sh->tokens[1], tokens_hi);
  }
  if (warp == 0) {
    int before = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 32) {
      const int b = b0 + lane;
      const int s = before + warp_scan(b < a.batch ? pref[b] : 0, lane);
      if (b < a.batch) pref[b] = s;
      before = __shfl_sync(0xffffffffu, s, 31);
    }
    if (lane == 0) sh->total = before;
  }
  __syncthreads();
  if (reports && threadIdx.x == 0 && overlapping(a, sh)) flag_error(a.err, KVQ_DEVERR_BAD_POS);
}

// A loop count that the compiler does not see through: loops that are to stay
// rolled were unrolled where it was a constant, pragma or not.
__device__ __forceinline__ int rolled(int n) {
  asm volatile("" : "+r"(n));
  return n;
}

// ---------------------------------------------------------------- unpacking
// binary16 pair of the codes at bits S (low half) and 16 + S (high half) of
// w, S + B <= 8: the code's bits dropped into the mantissa of 2^(10 - S) (whose
// last place is then worth 2^-S at bit 0, 1 at bit S), which is subtracted.
template <int B, int S>
__device__ __forceinline__ __half2 code_pair(uint32_t w) {
  constexpr uint32_t mask = ((1u << B) - 1) << S;
  constexpr uint32_t magic = 0x6400u - S * 0x400u;
  uint32_t x = (w & (mask | (mask << 16))) | (magic | (magic << 16));
  const uint32_t mm = magic | (magic << 16);
  return __hsub2(*reinterpret_cast<__half2*>(&x), *reinterpret_cast<const __half2*>(&mm));
}

// The same for field e (0 .. 16/B - 1) of the halves.
template <int B>
__device__ __forceinline__ __half2 code_field(uint32_t w, int e) {
  const int s = (B * e) & 7;
  if (B * e >= 8) w >>= 8;
  if constexpr (B == 8) {
    return code_pair<8, 0>(w);
  } else if constexpr (B == 4) {
    return s == 0 ? code_pair<4, 0>(w) : code_pair<4, 4>(w);
  } else {
    return s == 0   ? code_pair<2, 0>(w)
           : s == 2 ? code_pair<2, 2>(w)
           : s == 4 ? code_pair<2, 4>(w)
                    : code_pair<2, 6>(w);
  }
}

// The stored roundings of a group's scale and zero can push its largest value
// past binary16's range (65504).  Held in one piece, its scale then gives up
// last places, four at most (2^-8 of a range of 131008 at most, where the
// roundings are 2^-10); in two, the high one stops at 65504 and the low one
// has the rest (see value_pair).  Infinite parameters stay as they are.
template <int KP, int B, int N>
__device__ __forceinline__ void fit_range(uint32_t (&scale2)[N], const uint32_t (&zero2)[N]) {
  if constexpr (KP == 2) return;
  const __half2 top = __float2half2_rn(static_cast<float>((1 << B) - 1));
  auto largest = [&](int i) {
    return __hfma2(top, *reinterpret_cast<const __half2*>(&scale2[i]),
                   *reinterpret_cast<const __half2*>(&zero2[i]));
  };
  __half2 most = largest(0);
#pragma unroll
  for (int i = 1; i < N; ++i) most = __hmax2(most, largest(i));
  const uint32_t u = *reinterpret_cast<const uint32_t*>(&most);
  if ((u & 0xffffu) == 0x7c00u || (u >> 16) == 0x7c00u) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll 1
      for (int k = 0, kn = rolled(4); k < kn; ++k) {
        const __half2 t = largest(i);
        const uint32_t w = *reinterpret_cast<const uint32_t*>(&t);
        // the next binary16 scale towards zero
        auto over = [&](int s) {
          return ((w >> s) & 0xffffu) == 0x7c00u && ((scale2[i] >> s) & 0xffffu) != 0x7c00u &&
                 ((zero2[i] >> s) & 0xffffu) != 0x7c00u;
        };
        scale2[i] -= (over(0) ? 1u : 0u) + (over(16) ? 0x10000u : 0u);
      }
    }
  }
}

// hi and lo binary16 pairs of code * scale + zero, for two codes.
template <int KP>
__device__ __forceinline__ void value_pair(__half2 code, uint32_t scale2, uint32_t zero2,
                                           uint32_t& hi, uint32_t& lo) {
  if constexpr (KP == 1) {
    const __half2 v = __hfma2(code, *reinterpret_cast<__half2*>(&scale2),
                              *reinterpret_cast<__half2*>(&zero2));
    hi = *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const float2 c = __half22float2(code), s = unpack_half2(scale2), z = unpack_half2(zero2);
    const float x = fmaf(c.x, s.x, z.x), y = fmaf(c.y, s.y, z.y);
    // (65504 at most, see fit_range; infinities and NaN go on in lo)
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(y), "f"(x));
    const float2 h = unpack_half2(hi);
    lo = f2_to_h2(x - h.x, y - h.y);
  }
}

template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t* w) {
  if constexpr (N == 1) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    w[0] = u.x; w[1] = u.y;
  }
}

__device__ __forceinline__ void store_chunk(uint8_t* p, const uint32_t (&x)[4]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(x[0], x[1], x[2], x[3]);
}

// Place of a 16-byte chunk of key row r (of a ring block) among the row's
// D B / 128 chunks: exchanged so that the loads of eight rows' same chunk hit
// different banks.
__device__ __forceinline__ int key_chunk_swizzle(int chunks, int r) {
  return chunks >= 8 ? r & 7 : chunks == 4 ? (r >> 1) & 3 : chunks == 2 ? (r >> 2) & 1 : 0;
}

// Keys of one ring block into rows of the K tile: one lane a position (row r
// of the tile), elements [part * D / PARTS, + D / PARTS), 32 at a time in a
// short loop (see rolled; straight code for all of them was 3 to 7 % slower
// where few rows wait for the keys, 2 % faster at 2048 tokens).
template <class C, int B>
__device__ __forceinline__ void unpack_keys(const uint8_t* codes, const uint32_t* params,
                                            int gshift, int pos, int part, bool live,
                                            uint8_t* tile, int r) {
  constexpr int D = C::D, NS = D / 32 / C::PARTS;  // 32-element spans of this lane
  constexpr int LOAD = B == 8 ? 2 : 1;             // words of a slice in a span
  constexpr int E = 16 / B;
  const int groups = D >> gshift;
  const uint8_t* row = codes + pos * (D * B / 8);
  const int swz = key_chunk_swizzle(D * B / 128, pos) << 4;
  uint8_t* dst = tile + r * 128;
  const int rx = (r & 7) << 4;
#pragma unroll 1
  for (int i = 0, n = rolled(NS); i < n; ++i) {
    const int span = part * NS + i;
    uint32_t w[4][LOAD];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int off = c * (D * B / 32) + (span * B / 4) * 4;
      load_words<LOAD>(row + (((off & ~15) ^ swz) | (off & 15)), w[c]);
      if (B == 2) w[c][0] >>= (span & 1) * 8;
    }
    const uint32_t par = live ? params[pos * groups + (32 * span >> gshift)] : 0u;
    uint32_t scale2[1] = {__byte_perm(par, 0, 0x1010)}, zero2[1] = {__byte_perm(par, 0, 0x3232)};
    fit_range<C::KP, B>(scale2, zero2);
    uint8_t* half = dst + (span >> 1) * (C::NT * 128);  // 64 elements a swizzled row
    const int x0 = ((span & 1) << 6) ^ rx;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        value_pair<C::KP>(code_field<B>(w[c][e / E], e % E), scale2[0], zero2[0], hi[c], lo[c]);
      uint8_t* at = half + (x0 ^ (e << 4));
      store_chunk(at, hi);
      if constexpr (C::KP == 2) store_chunk(at + C::KPIECE, lo);
    }
  }
}

// Values of one ring block into columns of the V tile (its rows are elements,
// 64 positions a 128-byte row): lane = 8 octet + m takes the elements 8u + m
// of the octet's eight positions, u in [part * D/8 / PARTS, ...).
template <class C, int B>
__device__ __forceinline__ void unpack_values(const uint8_t* codes, const uint32_t* params,
                                              int gshift, int lane, int part, int live,
                                              uint8_t* tile, int octet0) {
  constexpr int D = C::D, NS = D / 32 / C::PARTS;
  constexpr int W = D * B / 128;                    // words of an octet in a format lane
  constexpr int N = D * B / 16, P = N < 16 ? N : 16;
  constexpr int LOAD = B == 8 ? 2 : 1;              // words of a 32-element span
  constexpr int E = 16 / B;
  const int groups = D >> gshift, inside = (1 << gshift) - 32;  // 32-element part in a group
  const int octet = lane >> 3, m = lane & 7;        // octet of the block: 0 .. 3
  const uint8_t* base = codes + (octet >> 1) * (2 * D * B) + 4 * m * P;
  const int og = octet0 + octet;                    // octet of the tile
  uint8_t* col = tile + (og >> 3) * (D * 128) + m * 128 + (((og & 7) ^ m) << 4);
  uint32_t scale2[4] = {0, 0, 0, 0}, zero2[4] = {0, 0, 0, 0};
#pragma unroll 1
  for (int i = 0, n = rolled(NS); i < n; ++i) {
    const int span = part * NS + i;
    uint32_t w[4][LOAD];
    const int nb = 4 * ((octet & 1) * W + span * B / 4);
    const uint8_t* src = base + (nb / P) * (32 * P) + nb % P;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      load_words<LOAD>(src + x * P, w[x]);
      if (B == 2) w[x][0] >>= (span & 1) * 8;
    }
    if (i == 0 || ((32 * span) & inside) == 0) {  // a group begins
      const uint32_t* par = params + (octet * 8) * groups + (32 * span >> gshift);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int k = octet * 8 + 2 * x;
        const uint32_t p0 = k < live ? par[(2 * x) * groups] : 0u;
        const uint32_t p1 = k + 1 < live ? par[(2 * x + 1) * groups] : 0u;
        scale2[x] = __byte_perm(p0, p1, 0x5410);
        zero2[x] = __byte_perm(p0, p1, 0x7632);
      }
      fit_range<C::KP, B>(scale2, zero2);
    }
    uint8_t* dst = col + span * (4 * 8 * 128);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int x = 0; x < 4; ++x)
        value_pair<C::KP>(code_field<B>(w[x][e / E], e % E), scale2[x], zero2[x], hi[x], lo[x]);
      store_chunk(dst + e * (8 * 128), hi);
      if constexpr (C::KP == 2) store_chunk(dst + e * (8 * 128) + C::KPIECE, lo);
    }
  }
}

// Positions that no row of the unit sees: zero, so that weights of 0 stay 0.
template <class C, bool KEYS>
__device__ __forceinline__ void zero_block(int lane, int part, uint8_t* tile, int blk) {
  constexpr int CU = C::D / 8 / C::PARTS;
  const uint32_t z[4] = {0, 0, 0, 0};
#pragma unroll 1
  for (int uu = 0, uun = rolled(CU); uu < uun; ++uu) {
    const int u = part * CU + uu;
    uint8_t* dst;
    if (KEYS) {
      const int r = blk * kBlock + lane;
      dst = tile + (u / 8) * (C::NT * 128) + r * 128 + (((u & 7) ^ (r & 7)) << 4);
    } else {
      const int og = blk * 4 + (lane >> 3), m = lane & 7;
      dst = tile + (og >> 3) * (C::D * 128) + (8 * u + m) * 128 + (((og & 7) ^ m) << 4);
    }
    store_chunk(dst, z);
    if (C::KP == 2) store_chunk(dst + C::KPIECE, z);
  }
}

// ------------------------------------------------------------------- roles
struct RingLayout {
  int bytes, k, v, kp, vp;  // block size; offsets of its four arrays
  int blocks;
};

__device__ __forceinline__ RingLayout ring_layout(const BlockCache& c, int avail) {
  RingLayout l;
  l.k = 0;
  l.v = kBlock * c.head_dim * c.bits_k / 8;
  l.kp = l.v + kBlock * c.head_dim * c.bits_v / 8;
  l.vp = l.kp + kBlock * (c.head_dim >> c.gshift_k) * 4;
  l.bytes = l.vp + kBlock * (c.head_dim >> c.gshift_v) * 4;
  // Whole turns of the copiers: each block is always filled by one warp, which
  // so never waits for a use that is two phases away (a phase bit would not
  // tell it from the one before).
  l.blocks = 0;
  while (l.blocks < kRing && (l.blocks + kCopiers) * l.bytes <= avail) l.blocks += kCopiers;
  return l;
}

// Work list (warp 25).
template <class C>
__device__ __forceinline__ bool list_role(const ChunkArgs& a, Shared* sh, const int* pref,
                                          const Waiter& wait) {
  const int lane = threadIdx.x & 31;
  const int Wu = overlapping(a, sh) ? 0 : sh->total;
  const long long W = static_cast<long long>(Wu) * a.c.kv_heads;
  long long share = (W + gridDim.x - 1) / gridDim.x;
  if (share < a.min_share) share = a.min_share;
  long long w = share * blockIdx.x;
  const long long w1 = min(W, w + share);
  int piece = 0;
  uint32_t headers = 0;  // partial slots that this CTA filled
  bool ok = true;
  if (w < w1) {
    int h = static_cast<int>(w / Wu);
    const int x0 = static_cast<int>(w - static_cast<long long>(h) * Wu);
    int b, lo = 0, hi = a.batch;  // first row whose inclusive prefix exceeds x0
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (pref[mid] > x0)
        hi = mid;
      else
        lo = mid + 1;
    }
    b = lo;
    RowInfo r = row_info(a, b);
    int within = x0 - (b > 0 ? pref[b - 1] : 0);
    int mt = (r.n * a.gq + C::UNIT - 1) / C::UNIT, m = 0;
    __syncwarp();
    while (true) {  // 32 units at a time
      const int c = m + lane < mt ? unit_cost<C>(a, r.n, r.len, m + lane) : 0;
      const int s = warp_scan(c, lane);
      const uint32_t above = __ballot_sync(0xffffffffu, s > within);
      if (above != 0) {
        const int f = __ffs(above) - 1;
        within -= __shfl_sync(0xffffffffu, s - c, f);
        m += f;
        break;
      }
      within -= __shfl_sync(0xffffffffu, s, 31);
      m += 32;
    }
    while (ok && w < w1) {
      const Unit u = unit_of<C>(a, r.n, r.len, m);
      // the share's part [within, upto) of the unit's cost; its first kUnitCost
      // carry no steps
      const int cost = a.whole_units ? 1 : u.steps + kUnitCost;
      const int upto = static_cast<int>(min(static_cast<long long>(cost), within + (w1 - w)));
      const int j = a.whole_units ? 0 : max(0, within - kUnitCost);
      const int je = a.whole_units ? u.steps : max(0, upto - kUnitCost);
      w += upto - within;
      within = 0;
      if (je > j) {  // publish the piece
        ok = wait(&sh->d_empty[piece & 1], ((piece >> 1) & 1) ^ 1);
        if (!ok) break;
        if (lane == 0) {
          Piece& p = sh->piece[piece & 1];
          p.valid = 1;
          p.b = b; p.h = h; p.start = r.start; p.n = r.n; p.len = r.len;
          p.row0 = u.row0; p.rows = u.rows; p.wide = u.wide; p.lim = u.lim;
          p.t0 = u.wide ? j : min(u.nt, 2 * j);
          p.t1 = u.wide ? min(u.nt, je) : min(u.nt, 2 * je);
          p.nt0 = u.nt0;
          p.j0 = j; p.j1 = je; p.begin = j == 0; p.end = je == u.steps;
          mbar_arrive(&sh->d_full[piece & 1]);
          if (!(p.begin && p.end)) {
            int* hd = a.ws_head + (blockIdx.x * 2 + p.begin) * 8;
            hd[0] = 1; hd[1] = r.start; hd[2] = h; hd[3] = u.row0; hd[4] = u.rows; hd[5] = p.end;
            headers |= 1u << p.begin;
          }
        }
        ++piece;
      }
      if (w < w1 && ++m == mt) {  // the next row with tokens
        m = 0;
        ++b;
        while (true) {
          if (b >= a.batch) {
            b = 0;
            ++h;
          }
          const int c = b + lane;
          const bool has = c < a.batch && row_info(a, c).n > 0;
          const uint32_t some = __ballot_sync(0xffffffffu, has);
          if (some != 0) {
            b += __ffs(some) - 1;
            break;
          }
          b += 32;
        }
        r = row_info(a, b);
        mt = (r.n * a.gq + C::UNIT - 1) / C::UNIT;
      }
    }
  }
  // the end of the list, and the partial slots that stay empty
  if (ok) ok = wait(&sh->d_empty[piece & 1], ((piece >> 1) & 1) ^ 1);
  if (lane == 0) {
    if (ok) {
      sh->piece[piece & 1].valid = 0;
      mbar_arrive(&sh->d_full[piece & 1]);
    }
    if (!a.whole_units) {
      if (!(headers & 1u)) a.ws_head[(blockIdx.x * 2 + 0) * 8] = 0;
      if (!(headers & 2u)) a.ws_head[(blockIdx.x * 2 + 1) * 8] = 0;
    }
  }
  __syncwarp();
  return ok;
}

__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Copies (warps 26-27, blocks in turn).
template <class C>
__device__ __forceinline__ bool copy_role(const ChunkArgs& a, Shared* sh, uint8_t* ring,
                                          const RingLayout& rl, const Waiter& wait) {
  const int lane = threadIdx.x & 31, id = (threadIdx.x >> 5) - kWarpCopy;
  const int kb = C::D * a.c.bits_k / 8, vb = C::D * a.c.bits_v / 8;
  const int gk = C::D >> a.c.gshift_k, gv = C::D >> a.c.gshift_v;
  // place of chunk 32 j + lane of the keys' rows of kb / 16 chunks, less 512 j
  // (32 chunks are whole rows; rows of 8 chunks come in fours, so that j's
  // lowest bit is bit 2 of the row)
  const uint32_t dk0 = (lane ^ key_chunk_swizzle(kb / 16, lane >> (__ffs(kb / 16) - 1))) << 4;
  const uint32_t dk1 = dk0 ^ (kb / 16 == 8 ? 4 << 4 : 0);
  int slot = 0, turn = 0;
  uint32_t phase = 0;
  for (int piece = 0;; ++piece) {
    if (!wait(&sh->d_full[piece & 1], (piece >> 1) & 1)) return false;
    const Piece& pd = sh->piece[piece & 1];
    if (!pd.valid) return true;
    const int b = pd.b, h = pd.h, first = pd.t0 * C::NT, last = min(pd.lim, pd.t1 * C::NT);
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh->d_empty[piece & 1]);
    int page = 0;  // the pages of 32 blocks are looked up at once
    for (int p = first, i = 0; p < last; p += kBlock, ++i) {
      if ((i & 31) == 0) {
        const int q = p + lane * kBlock;
        page = b;
        if (a.table != nullptr && q < last) {
          page = a.table[static_cast<size_t>(b) * a.pages_per_seq + (q >> a.page_shift)];
          if (page < 0 || page >= a.c.blocks) {
            flag_error(a.err, KVQ_DEVERR_BAD_PAGE);
            page = -1;
          }
        }
      }
      const int block = __shfl_sync(0xffffffffu, page, i & 31);
      if (turn == id) {
        if (!wait(&sh->ring_empty[slot], phase ^ 1)) return false;
        if (block < 0) {  // (that row's output is unspecified)
          mbar_arrive(&sh->ring_full[slot]);
        } else {
          const int local = a.table != nullptr ? p & ((1 << a.page_shift) - 1) : p;
          const int cnt = min(kBlock, (last - p + 15) & ~15);  // whole V tiles
          const size_t row =
              (static_cast<size_t>(block) * a.c.kv_heads + h) * a.c.block_tokens + local;
          const uint32_t base = smem_addr(ring + slot * rl.bytes), dst = base + lane * 16;
          const uint8_t* k = a.c.k_codes + row * kb + lane * 16;
          const uint8_t* v = a.c.v_codes + row * vb + lane * 16;
          // (unrolled: one base address each, so that no copy waits until the
          // one before has taken its address)
          const int nk = cnt * kb - lane * 16, nv = cnt * vb - lane * 16;
#pragma unroll
          for (int j = 0; j < C::D / 16; ++j)
            if (j * 512 < nk) copy16(base + (j & 1 ? dk1 : dk0) + j * 512, k + j * 512);
#pragma unroll
          for (int j = 0; j < C::D / 16; ++j)
            if (j * 512 < nv) copy16(dst + rl.v + j * 512, v + j * 512);
          if (lane * 16 < cnt * gk * 4)
            copy16(dst + rl.kp, reinterpret_cast<const uint8_t*>(a.c.k_params + row * gk) + lane * 16);
          if (lane * 16 < cnt * gv * 4)
            copy16(dst + rl.vp, reinterpret_cast<const uint8_t*>(a.c.v_params + row * gv) + lane * 16);
          // arrives for this lane when its copies are there
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                           smem_addr(&sh->ring_full[slot]))
                       : "memory");
        }
      }
      turn = turn + 1 == kCopiers ? 0 : turn + 1;
      if (++slot == rl.blocks) {
        slot = 0;
        phase ^= 1;
      }
    }
  }
}

// Unpacking (warps 16-23).
template <class C, bool KEYS, int B>
__device__ __forceinline__ bool unpack_role(const ChunkArgs& a, Shared* sh, uint8_t* tiles,
                                            const uint8_t* ring, const RingLayout& rl,
                                            const Waiter& wait) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int w = ((warp - kWarpUnpack) >> 2) * 2 + (warp & 1);  // of the role's four
  const int blk = w / C::PARTS, part = w % C::PARTS;
  uint64_t* full = KEYS ? sh->k_full : sh->v_full;
  uint64_t* empty = KEYS ? sh->k_empty : sh->v_empty;
  const int gshift = KEYS ? a.c.gshift_k : a.c.gshift_v;
  int slot = 0, tile = 0;
  uint32_t phase = 0;
  for (int piece = 0;; ++piece) {
    if (!wait(&sh->d_full[piece & 1], (piece >> 1) & 1)) return false;
    const Piece& p = sh->piece[piece & 1];
    if (!p.valid) return true;
    const int t0 = p.t0, t1 = p.t1, lim = p.lim;
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh->d_empty[piece & 1]);
    for (int t = t0; t < t1; ++t, ++tile) {
      const int used = min(C::BLOCKS, (lim - t * C::NT + kBlock - 1) / kBlock);
      uint8_t* dst = tiles + (tile & 1) * C::STAGE;
      if (!wait(&empty[tile & 1], ((tile >> 1) & 1) ^ 1)) return false;
      // A phase bit tells one use of a ring block from the next only: the use
      // before this one must be filled.  It is a block of an earlier tile
      // (the ring holds a tile), so with a short ring that tile is waited for.
      if (rl.blocks < 2 * C::BLOCKS && tile > 0 &&
          !wait(&full[(tile - 1) & 1], ((tile - 1) >> 1) & 1))
        return false;
      if (blk < used) {
        int s = slot + blk;
        uint32_t ph = phase;
        if (s >= rl.blocks) {
          s -= rl.blocks;
          ph ^= 1;
        }
        if (!wait(&sh->ring_full[s], ph)) return false;
        const uint8_t* src = ring + s * rl.bytes;
        const int live = lim - t * C::NT - blk * kBlock;  // positions of the block that are seen
        if constexpr (KEYS)
          unpack_keys<C, B>(src + rl.k, reinterpret_cast<const uint32_t*>(src + rl.kp), gshift,
                            lane, part, lane < live, dst, blk * kBlock + lane);
        else
          unpack_values<C, B>(src + rl.v, reinterpret_cast<const uint32_t*>(src + rl.vp), gshift,
                              lane, part, live, dst, blk * 4);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->ring_empty[s]);
      } else {
        zero_block<C, KEYS>(lane, part, dst, blk);
      }
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[tile & 1]);
      slot += used;
      while (slot >= rl.blocks) {
        slot -= rl.blocks;
        phase ^= 1;
      }
    }
  }
}

// MMA issue (warp 24; operands are uniform over the warp, one lane issues).
template <class C>
__device__ __forceinline__ void issue_scores(uint32_t s_tmem, uint32_t q, uint32_t k) {
  constexpr uint32_t idesc = tc::idesc_f16_kk(128, C::NT);
  const uint64_t q0 = tc::smem_desc_k128(q), k0 = tc::smem_desc_k128(k);
  bool accumulate = false;
  // (Q piece, K piece) products; small ones first
#pragma unroll 1
  for (int x = C::PIECES - 1; x >= 0; --x) {
    uint64_t qa = q0 + (x == 2 ? C::QTILE >> 4 : 0), ka = k0 + (x == 1 ? C::KPIECE >> 4 : 0);
#pragma unroll 1
    for (int i = 0, in = rolled(C::D / 64); i < in; ++i) {  // 64 elements: four steps of 16 in a swizzled row
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        tc::mma_f16_ss(s_tmem, qa + 2 * y, ka + 2 * y, idesc, accumulate);
        accumulate = true;
      }
      qa += (128 * 128) >> 4;
      ka += (C::NT * 128) >> 4;
    }
  }
}

template <class C>
__device__ __forceinline__ void issue_output(uint32_t o_tmem, uint32_t p_tmem, uint32_t v,
                                             bool accumulate) {
  constexpr uint32_t idesc = tc::idesc_f16_kk(128, C::D);
  const uint64_t v0 = tc::smem_desc_k128(v);
#pragma unroll 1
  for (int x = C::PIECES - 1; x >= 0; --x) {
    // the weights of each half of the positions start at that half's columns
    const uint32_t pa = p_tmem + (x == 2 ? C::NT / 4 : 0);
    const uint64_t va = v0 + (x == 1 ? C::KPIECE >> 4 : 0);
#pragma unroll
    for (int i = 0; i < C::NT / 16; ++i) {
      constexpr int HALF = C::NT / 32;  // steps of 16 positions in a half
      tc::mma_f16_ts(o_tmem, pa + (i / HALF) * (C::NT / 2) + (i % HALF) * 8,
                     va + (i / 4) * ((C::D * 128) >> 4) + (i % 4) * 2, idesc, accumulate);
      accumulate = true;
    }
  }
}

template <class C>
__device__ __forceinline__ bool mma_role(Shared* sh, uint32_t smem, uint32_t tmem,
                                         const Waiter& wait) {
  int tile0 = 0;  // tiles of the pieces before
  uint32_t p_phase = 0;  // bit s: slot s
  for (int piece = 0;; ++piece) {
    if (!wait(&sh->d_full[piece & 1], (piece >> 1) & 1)) return false;
    const Piece& pd = sh->piece[piece & 1];
    if (!pd.valid) return true;
    auto uniform = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
    const bool wide = uniform(pd.wide) != 0;
    const int t0 = uniform(pd.t0), t1 = uniform(pd.t1), j0 = uniform(pd.j0), j1 = uniform(pd.j1);
    const int nt0 = uniform(pd.nt0);
    if (tc::elect_one()) mbar_arrive(&sh->d_empty[piece & 1]);
    if (!wait(&sh->q_full, piece & 1)) return false;
    // The scores of a slot's next tile follow the output product of its last
    // one; step j0 - 1 stands for the start, where only scores are issued.
    int k_seen = t0, v_seen = t0;  // tiles waited for
#pragma unroll 1
    for (int j = j0 - 1; j < j1; ++j) {
#pragma unroll 1
      for (int s = 0, sn = rolled(2); s < sn; ++s) {
        // slot s works in step j on tile t, in step j + 1 on tile u
        const int t = wide ? j : 2 * j + s, u = wide ? j + 1 : t + 2;
        const int tend = wide && s == 0 ? min(t1, nt0) : t1;
        const uint32_t s_tmem = tmem + s * C::S_COL;
        const bool output = j >= j0 && t < tend;
        if (output) {
          if (!wait(&sh->p_full[s], (p_phase >> s) & 1)) return false;
          p_phase ^= 1u << s;
          const int i = tile0 + t - t0;
          if (t == v_seen) {
            if (!wait(&sh->v_full[i & 1], (i >> 1) & 1)) return false;
            ++v_seen;
          }
          tc::fence_after_sync();
          if (tc::elect_one()) {
            issue_output<C>(tmem + C::O_BASE + s * C::O_COL, s_tmem,
                            smem + C::SMEM_V + (i & 1) * C::STAGE, j > j0);
            if (!wide || s == 1) tc::commit(&sh->v_empty[i & 1]);
          }
        }
        if (j + 1 < j1 && u < tend) {
          const int i = tile0 + u - t0;
          if (u == k_seen) {
            if (!wait(&sh->k_full[i & 1], (i >> 1) & 1)) return false;
            ++k_seen;
          }
          tc::fence_after_sync();
          if (tc::elect_one()) {
            issue_scores<C>(s_tmem, smem + (wide && s == 1 ? C::QTILE : 0),
                            smem + C::SMEM_K + (i & 1) * C::STAGE);
            tc::commit(&sh->s_full[s]);
            if (!wide || s == 1) tc::commit(&sh->k_empty[i & 1]);
          }
        } else if (output) {
          if (tc::elect_one()) tc::commit(&sh->s_full[s]);  // the slot's output is complete
        }
        __syncwarp();
      }
    }
    tile0 += t1 - t0;
  }
}

// Half of the queries of a warp's 32 rows as binary16 (two pieces for PIECES 3), each
// row scaled by a power of two that brings its largest magnitude to
// [2^14, 2^15): bf16 and f16 rows stay exact down to 2^-28 of the largest
// element.  unscale[row] undoes it.  A row's elements are taken by D/8
// consecutive lanes, several rows at once: with a row per lane the loads of a
// warp touched 32 lines each and took 11000 cycles a unit.  off, valid: of
// this lane's own row, row0 + lane.
template <class C, bool ROT>
__device__ __forceinline__ void load_queries(const ChunkArgs& a, size_t off, bool valid,
                                             uint8_t* q, float* unscale, int row0, int half) {
  constexpr int D = C::D, LANES = D / 8, ROWS = 32 / LANES;  // of a row; rows at once
  const int lane = threadIdx.x & 31, u = lane % LANES;
  const bool f32 = a.q_dtype == KVQ_F32;
  const int turns = f32 || LANES < 16 ? 4 : 8;  // eight loads at a time, at most
  const uint32_t kinds = __ballot_sync(0xffffffffu, valid);
#pragma unroll 1
  for (int t0 = half * LANES / 2; t0 < (half + 1) * LANES / 2; t0 += turns) {
    uint4 raw[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = ((t0 + (f32 ? i / 2 : i)) * ROWS + lane / LANES) & 31;
      const size_t at = __shfl_sync(0xffffffffu, off, row) + 8 * u;
      raw[i] = make_uint4(0, 0, 0, 0);
      if ((kinds >> row) & 1)
        raw[i] = f32 ? reinterpret_cast<const uint4*>(static_cast<const float*>(a.q) + at)[i & 1]
                     : *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + at);
    }
#pragma unroll 1
    for (int t = t0; t < t0 + turns; ++t) {
      float x[8];
      const uint32_t w[8] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w,
                             raw[1].x, raw[1].y, raw[1].z, raw[1].w};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t h = k & 1 ? w[k / 2] >> 16 : w[k / 2] & 0xffffu;
        x[k] = f32                      ? __uint_as_float(w[k])
               : a.q_dtype == KVQ_BF16 ? __uint_as_float(h << 16)
                                       : __half2float(__ushort_as_half(static_cast<uint16_t>(h)));
      }
#pragma unroll
      for (int i = 0; i < 7; ++i) raw[i] = f32 && i < 6 ? raw[i + 2] : raw[i + 1];
      if constexpr (ROT) {  // H q / D, the butterfly h = 1, 2, ..., D/2
#pragma unroll
        for (int h = 1; h < 8; h *= 2)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if ((i & h) == 0) {
              const float y = x[i], z = x[i + h];
              x[i] = y + z;
              x[i + h] = y - z;
            }
#pragma unroll
        for (int m = 1; m < LANES; m *= 2)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float y = __shfl_xor_sync(0xffffffffu, x[i], m);
            x[i] = u & m ? y - x[i] : y + x[i];
          }
      }
      float amax = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fabsf(x[k]));
#pragma unroll
      for (int m = 1; m < LANES; m *= 2) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
      const int e = max(static_cast<int>((__float_as_uint(amax) >> 23) & 0xff) - 127 - 14, -126);
      const float up = pow2i(-e);  // e <= 114
      const int r = row0 + t * ROWS + lane / LANES;
      if (u == 0) unscale[r] = pow2i(e) * (ROT ? 1.0f / D : 1.0f);
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float y0 = x[2 * c] * up, y1 = x[2 * c + 1] * up;
        hi[c] = f2_to_h2(y0, y1);
        if constexpr (C::PIECES == 3) {
          const float2 h = unpack_half2(hi[c]);
          lo[c] = f2_to_h2(y0 - h.x, y1 - h.y);
        }
      }
      uint8_t* dst = q + (u / 8) * (128 * 128) + r * 128 + (((u & 7) ^ (r & 7)) << 4);
      store_chunk(dst, hi);
      if constexpr (C::PIECES == 3) store_chunk(dst + C::QTILE, lo);
    }
  }
}

// Eight consecutive output elements.
__device__ __forceinline__ void store_out8(void* out, int dtype, size_t i, const float (&x)[8]) {
  if (dtype == KVQ_F32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(out) + i);
    p[0] = make_float4(x[0], x[1], x[2], x[3]);
    p[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (dtype == KVQ_BF16) {
        __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * c], x[2 * c + 1]);
        w[c] = *reinterpret_cast<uint32_t*>(&h);
      } else {
        w[c] = f2_to_h2(x[2 * c], x[2 * c + 1]);
      }
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + i) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Two binary32 values side by side (packed operations of sm_100).
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}

// Weights 2^(s c + shift) of two scores, rounded to binary16 (p; q: the rest of
// the rounding, for three pieces), and their sums in binary32 (sum2).
template <int PIECES>
__device__ __forceinline__ void weights(uint32_t u, uint32_t v, uint64_t c2, uint64_t shift2,
                                        uint64_t& sum2, uint32_t& p, uint32_t& q) {
  uint64_t s;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(s)
      : "l"(pair(__uint_as_float(u), __uint_as_float(v))), "l"(c2), "l"(shift2));
  float x, y;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(s));
  x = exp2_approx(x);
  y = exp2_approx(y);
  asm("add.rn.f32x2 %0, %0, %1;" : "+l"(sum2) : "l"(pair(x, y)));
  p = f2_to_h2(x, y);
  if constexpr (PIECES == 3) {
    const float2 h = unpack_half2(p);
    q = f2_to_h2(x - h.x, y - h.y);
  }
}

__device__ __forceinline__ float sum_of(uint64_t s) {
  float x, y;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(s));
  return x + y;
}

// Softmax (warps 0-7: slot 0, 8-15: slot 1).  A thread has one row and half of a
// tile's columns, as of the output's elements: with whole rows a slot's tile
// took twice as long, and between two products of a slot lies its softmax.
// The two warps of 32 rows agree on the maxima through shared memory.
template <class C, bool ROT>
__device__ __forceinline__ bool softmax_role(const ChunkArgs& a, Shared* sh, uint8_t* smem,
                                             uint32_t tmem, const Waiter& wait) {
  constexpr int D = C::D, NH = C::NT / 2, DH = D / 2;  // this thread's columns
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int slot = warp >> 3, half = (warp >> 2) & 1, quarter = warp & 3;
  const int r = quarter * 32 + lane;  // row of the slot
  const uint32_t quad = static_cast<uint32_t>(quarter * 32) << 16;
  const uint32_t s_tmem = tmem + quad + slot * C::S_COL + half * NH;
  const uint32_t o_tmem = tmem + quad + C::O_BASE + slot * C::O_COL + half * DH;
  uint32_t s_phase = 0, merges = 0, turn = 0;
  // Exchange of a value with the row's other thread.  Two turns' places: a
  // warp that is a turn ahead does not overwrite what the other still reads.
  auto other_half = [&](float mine, float& theirs) {
    sh->top[slot][turn & 1][half][r] = mine;
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh->x_full[slot][quarter]);
    if (!wait(&sh->x_full[slot][quarter], turn & 1)) return false;
    theirs = sh->top[slot][turn & 1][half ^ 1][r];
    ++turn;
    return true;
  };
  for (int piece = 0;; ++piece) {
    if (!wait(&sh->d_full[piece & 1], (piece >> 1) & 1)) return false;
    const Piece& pd = sh->piece[piece & 1];
    if (!pd.valid) return true;
    const bool wide = pd.wide;
    const int t0 = pd.t0, t1 = pd.t1, nt0 = pd.nt0, j0 = pd.j0;
    const int rows = pd.rows, ur = wide ? slot * 128 + r : r;  // row of the unit
    const bool valid = ur < rows;
    const bool whole = pd.begin && pd.end;
    const int br = pd.row0 + (valid ? ur : 0);                 // row of the batch row
    const int token = pd.start + br / a.gq, head = pd.h * a.gq + br % a.gq;
    const int limit = valid ? limit_of(a, pd.n, pd.len, br) : 0x7fffffff;
    const int part = pd.begin;
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh->d_empty[piece & 1]);
    // the slot's tiles of this piece: t, t + stride, ... < tend
    int t, tend, stride;
    if (wide) {
      t = t0; tend = slot == 0 ? min(t1, nt0) : t1; stride = 1;
    } else {
      t = 2 * j0 + slot; tend = t1; stride = 2;
    }
    const bool any_tile = t < tend;
    const bool works = __any_sync(0xffffffffu, valid);  // warps without rows only keep pace
    // ---- queries (a narrow unit's slot 1 has the rows of slot 0)
    if ((wide || slot == 0) && works) {
      load_queries<C, ROT>(
          a, static_cast<size_t>(token) * a.q_stride + static_cast<size_t>(head) * D, valid,
          smem + (wide ? slot * C::QTILE : 0), sh->unscale[wide ? slot : 0], quarter * 32, half);
      fence_proxy_async_shared();
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh->q_full);
    if (!wait(&sh->q_full, piece & 1)) return false;
    const float unscale = works ? sh->unscale[wide ? slot : 0][r] : 1.0f;
    // scores in units of log2: S * c
    const float c = fmaxf(a.sm_scale_log2 * unscale, 1.2e-38f);
    float m = -INFINITY, l = 0.0f;
    for (bool first = true; t < tend; t += stride, first = false) {
      if (!wait(&sh->s_full[slot], s_phase)) return false;
      s_phase ^= 1;
      tc::fence_after_sync();
      if (works) {
        const int seen = limit - t * C::NT - half * NH;
        if (__any_sync(0xffffffffu, seen < NH)) {  // masked: -inf in place
#pragma unroll 1
          for (int i = 0, in = rolled(NH / 16); i < in; ++i) {
            uint32_t s[16];
            tc::ld_32x32b<16>(s_tmem + 16 * i, s);
            tc::wait_ld(s);
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if (16 * i + k >= seen) s[k] = 0xff800000u;
            tc::st_32x32b_x16(s_tmem + 16 * i, s);
          }
          tc::wait_st();
        }
        // The scores are read twice, for their maximum and for the weights, 16 at
        // a time in short loops: held in registers, or with the next 16 on their
        // way, the longer code costs more than it hides.
        float mx;
        {
          float top[4] = {m, -INFINITY, -INFINITY, -INFINITY};  // (a chain each)
#pragma unroll 1
          for (int i = 0, in = rolled(NH / 16); i < in; ++i) {
            uint32_t s[16];
            tc::ld_32x32b<16>(s_tmem + 16 * i, s);
            tc::wait_ld(s);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              top[k & 3] = fmaxf(top[k & 3], fmaxf(__uint_as_float(s[2 * k]),
                                                   __uint_as_float(s[2 * k + 1])));
          }
          float theirs;
          mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
          if (!other_half(mx, theirs)) return false;
          mx = fmaxf(mx, theirs);
        }
        if (first) {
          m = mx;
        } else if (__any_sync(0xffffffffu, (mx - m) * c > C::kThreshold)) {
          // (false while nothing is seen; the same in both warps) every row
          // moves to its maximum, and its sums follow
          const float f = mx == -INFINITY ? 1.0f : exp2_approx((m - mx) * c);
          l *= f;
          m = mx;
#pragma unroll 1
          for (int i = 0, in = rolled(DH / 16); i < in; ++i) {
            uint32_t o[16];
            tc::ld_32x32b<16>(o_tmem + 16 * i, o);
            tc::wait_ld(o);
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
            tc::st_32x32b_x16(o_tmem + 16 * i, o);
          }
        }
        const float shift = C::kOffset - (m == -INFINITY ? 0.0f : m * c);
        const uint64_t c2 = pair(c, c), shift2 = pair(shift, shift);
        uint64_t sum2[2] = {0, 0};
        if constexpr (C::PIECES < 3) {
          // (a chunk's weights take columns that were read)
#pragma unroll 1
          for (int i = 0, in = rolled(NH / 16); i < in; ++i) {
            uint32_t s[16], p[8];
            tc::ld_32x32b<16>(s_tmem + 16 * i, s);
            tc::wait_ld(s);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              uint32_t none;
              weights<C::PIECES>(s[2 * k], s[2 * k + 1], c2, shift2, sum2[k & 1], p[k], none);
            }
            tc::st_32x32b_x8(s_tmem + 8 * i, p);
          }
        } else {
          // two binary16 pieces take a score's column each: all scores are
          // read before the first are written
          static_assert(C::PIECES < 3 || NH == 32, "the scores of half a tile in two loads");
          uint32_t s[2][16];
          tc::ld_32x32b<16>(s_tmem, s[0]);
          tc::ld_32x32b<16>(s_tmem + 16, s[1]);
          tc::wait_ld(s[0]);
          tc::wait_ld(s[1]);
          uint32_t p[16], q[16];
#pragma unroll
          for (int k = 0; k < 16; ++k)
            weights<3>(s[k / 8][2 * (k % 8)], s[k / 8][2 * (k % 8) + 1], c2, shift2, sum2[k & 1],
                       p[k], q[k]);
          tc::st_32x32b_x16(s_tmem, p);
          tc::st_32x32b_x16(s_tmem + NH / 2, q);
        }
        l += sum_of(sum2[0]) + sum_of(sum2[1]);
        tc::wait_st();
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->p_full[slot]);
    }
    // ---- the slot's output
    if (any_tile) {
      if (!wait(&sh->s_full[slot], s_phase)) return false;
      s_phase ^= 1;
      tc::fence_after_sync();
    }
    if (works) {  // the row's whole sum
      float theirs;
      if (!other_half(l, theirs)) return false;
      l = half == 0 ? l + theirs : theirs + l;
    }
    float f0 = 1.0f, f1 = 0.0f;
    // slot 1's row (this half of it), swizzled
    float4* merge = reinterpret_cast<float4*>(smem) + r * (D / 4) + half * (DH / 4);
    const bool other = !wide && 2 * j0 + 1 < t1;  // slot 1 has an output
    if (!wide) {
      if (slot == 1) {
        if (other && works) {
#pragma unroll 1
          for (int i = 0, in = rolled(DH / 16); i < in; ++i) {
            uint32_t o[16];
            tc::ld_32x32b<16>(o_tmem + 16 * i, o);
            tc::wait_ld(o);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              merge[(4 * i + k) ^ (r & 7)] =
                  make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]),
                              __uint_as_float(o[4 * k + 2]), __uint_as_float(o[4 * k + 3]));
          }
        }
        if (half == 0) sh->stat[r] = make_float2(m, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->m_full);
      } else {
        if (!wait(&sh->m_full, merges & 1)) return false;
        const float2 st = sh->stat[r];
        const float mm = fmaxf(m, st.x), base = mm == -INFINITY ? 0.0f : mm;
        f0 = exp2_approx((m - base) * c);
        f1 = exp2_approx((st.x - base) * c);
        l = l * f0 + st.y * f1;
        m = mm;
      }
    }
    if ((wide || slot == 0) && works) {
      // A row that sees no position yields 0.  Any other sum is divided by, so
      // that NaN, and scores of -inf alone, come out as the quotient's NaN.
      const bool nothing = whole && limit <= 0;
      if (whole) {
        const float inv = nothing ? 0.0f : 1.0f / l;
        f0 *= inv;
        f1 *= inv;
      }
      // the row's place in the output, or among the partial results
      const size_t prow = static_cast<size_t>(blockIdx.x * 2 + part) * a.part_rows + ur;
      if (!whole && valid && half == 0)
        a.ws_ml[prow] = make_float2(m == -INFINITY ? m : m * c, limit <= 0 ? -1.0f : l);
      const int type = whole ? a.out_dtype : static_cast<int>(KVQ_F32);
      const size_t row = whole ? (static_cast<size_t>(token) * a.q_heads + head) * D : prow * D;
      const int es = type == KVQ_F32 ? 4 : 2;
      uint8_t* dst = (whole ? static_cast<uint8_t*>(a.out) : reinterpret_cast<uint8_t*>(a.ws_o)) +
                     (row + half * DH) * es;
      // A wide unit's rows go through the slot's query tile, 16 columns at a
      // time, so that a store covers whole sectors of many rows.
      uint8_t* stage = smem + slot * C::QTILE + (quarter * 2 + half) * (C::QTILE / 8);
      const uint32_t rows_valid = __ballot_sync(0xffffffffu, valid);
#pragma unroll 1
      for (int i = 0, in = rolled(DH / 16); i < in; ++i) {
        uint32_t o[16];
        if (any_tile) {
          tc::ld_32x32b<16>(o_tmem + 16 * i, o);
          tc::wait_ld(o);
        } else {
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] = 0;
        }
        const int cs = es == 4 ? 2 : 1;  // log2 of 16-byte chunks in 16 columns
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(o[8 * k + e]) * f0;
          if (other) {
            const float4 y = merge[(4 * i + 2 * k) ^ (r & 7)];
            const float4 z = merge[(4 * i + 2 * k + 1) ^ (r & 7)];
            x[0] = fmaf(y.x, f1, x[0]); x[1] = fmaf(y.y, f1, x[1]);
            x[2] = fmaf(y.z, f1, x[2]); x[3] = fmaf(y.w, f1, x[3]);
            x[4] = fmaf(z.x, f1, x[4]); x[5] = fmaf(z.y, f1, x[5]);
            x[6] = fmaf(z.z, f1, x[6]); x[7] = fmaf(z.w, f1, x[7]);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = nothing ? 0.0f : x[e];
          if (wide) {  // rows of 64 bytes; chunk c of row r at c ^ (r / 2 mod 4)
            const int sw = (lane >> 1) & 3;
            if (es == 4) {
              float4* d = reinterpret_cast<float4*>(stage + lane * 64);
              d[(2 * k) ^ sw] = make_float4(x[0], x[1], x[2], x[3]);
              d[(2 * k + 1) ^ sw] = make_float4(x[4], x[5], x[6], x[7]);
            } else {
              store_out8(stage, type, (lane * 64 + ((k ^ sw) << 4)) / 2, x);
            }
          } else if (valid) {
            store_out8(dst, type, 16 * i + 8 * k, x);
          }
        }
        if (wide) {
          __syncwarp();
#pragma unroll 2
          for (int y = lane; y < 32 << cs; y += 32) {
            const int rr = y >> cs, ch = y & ((1 << cs) - 1);
            const uint4 v = *reinterpret_cast<const uint4*>(stage + rr * 64 +
                                                            ((ch ^ ((rr >> 1) & 3)) << 4));
            uint8_t* to = reinterpret_cast<uint8_t*>(
                __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), rr));
            if ((rows_valid >> rr) & 1)
              *reinterpret_cast<uint4*>(to + (((i << cs) + ch) << 4)) = v;
          }
          __syncwarp();
        }
      }
    }
    tc::fence_before_sync();
    // the rows on their way to the output lie in the query tiles' memory
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh->m_free);
    if (!wait(&sh->m_free, piece & 1)) return false;
    if (!wide) ++merges;
  }
}

template <class C, bool ROT>
__global__ void __launch_bounds__(kThreads, 1) chunk_kernel(const ChunkArgs a) {
  // (the swizzled tiles want 1024-byte boundaries; a pointer rounded up here
  // would lose its address space, and every access become a generic one)
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* ring = smem + C::SMEM_RING;
  Shared* sh = reinterpret_cast<Shared*>(smem + kSmemMax - kHeader);
  const RingLayout rl = ring_layout(a.c, kSmemMax - kHeader - C::SMEM_RING);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh->k_full[i], 4);
      mbar_init(&sh->k_empty[i], 1);
      mbar_init(&sh->v_full[i], 4);
      mbar_init(&sh->v_empty[i], 1);
      mbar_init(&sh->s_full[i], 1);
      mbar_init(&sh->p_full[i], 8);
      mbar_init(&sh->d_full[i], 1);
      mbar_init(&sh->d_empty[i], 25 + kCopiers);  // softmax 16, keys 4, values 4, MMA 1, copies
    }
    mbar_init(&sh->q_full, 16);
    mbar_init(&sh->m_full, 8);
    mbar_init(&sh->m_free, 16);
    mbar_init(&sh->drained, 1);
    for (int i = 0; i < 8; ++i) mbar_init(&sh->x_full[i >> 2][i & 3], 2);
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&sh->ring_full[i], blockIdx.x == 0 && i == a.fault_stage ? 33 : 32);
      mbar_init(&sh->ring_empty[i], 2 * C::PARTS);
    }
    sh->abort = 0;
    sh->tokens[0] = sh->tokens[1] = 0;
    fence_barrier_init();
  }
  if (warp == kWarpMma) {
    tc::alloc(&sh->tmem, 512);
    tc::relinquish();
  }
  pdl_wait();
  pdl_trigger();
  int* pref = reinterpret_cast<int*>(smem);  // (the tiles' memory is not yet in use)
  scan_rows<C>(a, pref, sh);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sh->tmem;
  const Waiter wait{&sh->abort, a.wait_limit_ns};

  if (warp < kWarpUnpack) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    softmax_role<C, ROT>(a, sh, smem, tmem, wait);
  } else if (warp < kWarpMma) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsUnpack));
    if ((warp & 2) == 0) {
      uint8_t* tiles = smem + C::SMEM_K;
      if (a.c.bits_k == 2)
        unpack_role<C, true, 2>(a, sh, tiles, ring, rl, wait);
      else if (a.c.bits_k == 4)
        unpack_role<C, true, 4>(a, sh, tiles, ring, rl, wait);
      else
        unpack_role<C, true, 8>(a, sh, tiles, ring, rl, wait);
    } else {
      uint8_t* tiles = smem + C::SMEM_V;
      if (a.c.bits_v == 2)
        unpack_role<C, false, 2>(a, sh, tiles, ring, rl, wait);
      else if (a.c.bits_v == 4)
        unpack_role<C, false, 4>(a, sh, tiles, ring, rl, wait);
      else
        unpack_role<C, false, 8>(a, sh, tiles, ring, rl, wait);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    if (warp == kWarpMma) {
      mma_role<C>(sh, smem_addr(smem), __shfl_sync(0xffffffffu, tmem, 0), wait);
    } else if (warp == kWarpList) {
      list_role<C>(a, sh, pref, wait);
    } else {
      copy_role<C>(a, sh, ring, rl, wait);
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kWarpMma) {
    tc::fence_after_sync();
    if (sh->abort != 0) {
      if ((threadIdx.x & 31) == 0) flag_error(a.err, KVQ_DEVERR_TIMEOUT);
      // products in flight end before their memory is given back (a commit
      // covers those of the thread that makes it: the one that issued them)
      if (tc::elect_one()) tc::commit(&sh->drained);
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(&sh->drained, 0) && global_timer_ns() - t0 < 10000000ull) {
      }
      __syncwarp();
    }
    tc::dealloc(tmem, 512);
  }
}

}  // namespace chunk
}  // namespace kvq
