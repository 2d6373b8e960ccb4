// Ragged quantize-and-append and its read-back (kvq_quantize_append_ragged,
// kvq_dequantize_ragged): packed tokens of rows of any lengths, each 16-position
// tile that takes tokens named by one entry of the slot map.
//
// One CTA handles one entry of one kv head, keys or values.  A thread owns two
// units of 8 consecutive elements of one token, the D/16 threads of a row in
// consecutive lanes.  Bits and group sizes are runtime values (uniform over
// the launch); the codes come from the same binary32 steps as in quantize.cuh,
//   mn, mx = group min and max (xor-shuffles over the group's lanes);
//   scale = (mx - mn) / (2^b - 1);  inv = 1 / scale;
//   code = rint((x - mn) * inv), 0 for a degenerate group,
// rint by adding 1.5 * 2^23, whose sum's low mantissa bits are the code.  Both
// layouts keep a unit's codes at one place of a word: element d = 8u + m
// (unit u, m = 0..7) sits at bit 16 (m mod 2) + b (u mod E) of
//   keys:   word u/E of slice m/2 of its row,
//   values: (position k of the tile) half k mod 2 of word (k/8) W + u/E of
//           lane 4m + (k mod 8)/2 (bit offset without the 16 (m mod 2)),
// E = 16/b, so a register per slice holds elements 2c and 2c+1 in its halves,
// shifted by b (u mod E); an or over the word's lanes completes it (the
// fields are disjoint).
//
// Bound: HBM traffic for long chunks (2 D es bytes in, D (bk + bv) / 8 + 4
// (D/Gk + D/Gv) out per token and head), launch latency for single tokens.
// Whole tiles are assembled in shared memory and leave as 16-byte stores; an
// edge tile's words go to global memory one by one, so that positions of no
// entry keep their bytes.  For 8200 tokens of 8 heads, head_dim 128,
// K4V2, on B200: append 16.3 us (2.5 TB/s in and out, 77 % of issue slots),
// read-back 11.1 us; with one unit a thread 39 and 24 us, since the group's
// exchanges and quotients are per thread.
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "serve.h"

namespace kvq {
namespace {

// Entry e of the map if it names places inside the cache and the packed
// tokens; count 0 (and an error flag) otherwise.
__device__ __forceinline__ int4 load_entry(const RaggedArgs& a, int e) {
  int4 m = a.map[e];  // (coherent: the planner may be the kernel before)
  if (m.w == 0) return m;
  uint32_t bad = 0;
  if (m.x < 0 || m.x >= a.c.blocks) bad |= KVQ_DEVERR_BAD_PAGE;
  if (m.y < 0 || m.w < 0 || m.w > 16 || (m.y & 15) + m.w > 16 || m.y >= a.c.block_tokens)
    bad |= KVQ_DEVERR_CAPACITY;
  if (m.z < 0 || m.z > a.num_tokens - m.w) bad |= KVQ_DEVERR_BAD_POS;
  if (bad) {
    if (threadIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) flag_error(a.err, bad);
    m.w = 0;
  }
  return m;
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]);
template <>
__device__ __forceinline__ void store8<float>(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
template <>
__device__ __forceinline__ void store8<__half>(__half* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(f2_to_h2(x[0], x[1]), f2_to_h2(x[2], x[3]),
                                            f2_to_h2(x[4], x[5]), f2_to_h2(x[6], x[7]));
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* p, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Walsh-Hadamard butterfly h = 1, 2, ..., D/2 of a row whose elements 16 t ..
// 16 t + 15 are in lane t: stages below 16 inside the thread, the others by
// xor-shuffles.
template <int D>
__device__ __forceinline__ void rotate_row(float (&x)[16], int t) {
#pragma unroll
  for (int h = 1; h < 16; h *= 2)
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if ((i & h) == 0) {
        const float p = x[i], q = x[i + h];
        x[i] = __fadd_rn(p, q);
        x[i + h] = __fsub_rn(p, q);
      }
#pragma unroll
  for (int m = 1; m < D / 16; m *= 2) {
    const bool upper = (t & m) != 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float y = __shfl_xor_sync(0xffffffffu, x[i], m);
      x[i] = upper ? __fsub_rn(y, x[i]) : __fadd_rn(x[i], y);
    }
  }
}

// log2 of the bytes of a format lane's piece, min(16, D b / 16).
__device__ __forceinline__ int v_piece_shift(int D, int b) { return D * b < 256 ? 3 : 4; }

// Byte offset of a value word's half of element 8u, position k, in a tile;
// element 8u + m lies 4 m pieces on.
__device__ __forceinline__ uint32_t v_half_offset(int D, uint32_t b, uint32_t k, uint32_t u) {
  const int ps = v_piece_shift(D, b);
  const uint32_t n = 4 * ((k >> 3) * (D * b >> 7) + (u * b >> 4)) + 2 * (k & 1);
  return ((n >> ps) << (ps + 5)) + (((k & 7) >> 1) << ps) + (n & ((1u << ps) - 1));
}

// 16 elements widened to binary32, by coherent loads (the read-back may be the
// kernel before).
template <typename T>
__device__ __forceinline__ void load16(const T* p, float (&x)[16]) {
  constexpr int N = static_cast<int>(sizeof(T));  // 16-byte loads
  uint4 u[N];
#pragma unroll
  for (int i = 0; i < N; ++i) u[i] = reinterpret_cast<const uint4*>(p)[i];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (std::is_same<T, float>::value) {
        x[4 * i + k] = __uint_as_float(w[k]);
      } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        x[8 * i + 2 * k] = __uint_as_float(w[k] << 16);
        x[8 * i + 2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
      } else {
        const float2 f = unpack_half2(w[k]);
        x[8 * i + 2 * k] = f.x;
        x[8 * i + 2 * k + 1] = f.y;
      }
    }
  }
}

template <int D, typename TIn, bool ROT>
__global__ void __launch_bounds__(D) append_ragged_kernel(const RaggedArgs a) {
  constexpr int U = D / 16;  // threads of a row
  __shared__ __align__(16) uint8_t codes[16 * D];  // a tile at 8 bits
  __shared__ __align__(16) uint32_t params[16 * (D / 32)];
  pdl_wait();
  pdl_trigger();
  const int4 e = load_entry(a, blockIdx.x);
  if (e.w == 0) return;
  const int h = blockIdx.y;
  const bool is_v = blockIdx.z != 0;
  const int b = is_v ? a.c.bits_v : a.c.bits_k, gshift = is_v ? a.c.gshift_v : a.c.gshift_k;
  const uint32_t t = threadIdx.x % U;  // thread of the row
  const int r = threadIdx.x / U;       // row of the tile
  const int first = e.y & 15;
  const bool full = e.w == 16;
  const bool valid = r >= first && r < first + e.w;
  const size_t row0 =
      (static_cast<size_t>(e.x) * a.c.kv_heads + h) * a.c.block_tokens + (e.y & ~15);

  float x[16];
  if (valid) {
    const TIn* src = static_cast<const TIn*>(is_v ? a.v : a.k) +
                     static_cast<int64_t>(e.z + r - first) * (is_v ? a.v_stride : a.k_stride) +
                     h * D + 16 * t;
    load16(src, x);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = 0.0f;
  }
  if (ROT && !is_v) rotate_row<D>(x, t);

  float mn = x[0], mx = x[0];
#pragma unroll
  for (int i = 1; i < 16; ++i) {
    mn = fminf(mn, x[i]);
    mx = fmaxf(mx, x[i]);
  }
  const int lanes = 1 << (gshift - 4);  // threads of a group: 2, 4 or 8
  for (int m = 1; m < lanes; m <<= 1) {
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, m));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, m));
  }
  mn = (mn == 0.0f) ? 0.0f : mn;  // a zero extreme is stored as +0
  mx = (mx == 0.0f) ? 0.0f : mx;
  const uint32_t levels = (1u << b) - 1;
  const float scale = __fdiv_rn(__fsub_rn(mx, mn), static_cast<float>(levels));
  const float inv = __frcp_rn(scale);
  const bool flat = scale == 0.0f || !isfinite(scale) || !isfinite(inv);
  const float f = flat ? 0.0f : inv, z = flat ? 0.0f : mn;
  // word c: elements 2c, 2c + 1 of both units, from bit b (u mod E)
  const int e1 = b == 2 ? 7 : b == 4 ? 3 : 1;  // E - 1
  const int shift = b * (2 * t & e1);
  uint32_t w[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float d = __fmul_rn(__fsub_rn(x[(i >> 1) * 8 + 2 * c + (i & 1)], z), f);
      q[i] = __float_as_uint(__fadd_rn(d, 12582912.0f)) & levels;  // 1.5 * 2^23
    }
    w[c] = ((q[0] | (q[1] << 16)) | ((q[2] | (q[3] << 16)) << b)) << shift;
  }
  for (int m = 2; m <= e1; m <<= 1) {  // lanes of a word: (e1 + 1) / 2
#pragma unroll
    for (int c = 0; c < 4; ++c) w[c] |= __shfl_xor_sync(0xffffffffu, w[c], m >> 1);
  }

  // the word's first lane stores it; the group's first lane its parameters
  const bool word_lane = (2 * t & e1) == 0, group_lane = (t & (lanes - 1)) == 0;
  const uint32_t par = pack_half2(__float2half_rn(scale), __float2half_rn(mn));
  const uint32_t row_bytes = D * b >> 3, groups = D >> gshift;
  uint8_t* gcodes = (is_v ? a.c.v_codes : a.c.k_codes) + row0 * row_bytes;  // (a tile: 16 rows)
  uint32_t* gparams = (is_v ? a.c.v_params : a.c.k_params) + row0 * groups;
  uint8_t* cdst = full ? codes : gcodes;
  uint32_t* pdst = full ? params : gparams;
  if (valid) {
    if (word_lane) {
      if (!is_v) {
        uint8_t* row = cdst + r * row_bytes + 4 * (t * b >> 3);
#pragma unroll
        for (int c = 0; c < 4; ++c)
          *reinterpret_cast<uint32_t*>(row + c * (row_bytes >> 2)) = w[c];
      } else {
        const int P = 1 << v_piece_shift(D, b);
        uint8_t* at = cdst + v_half_offset(D, b, r, 2 * t);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          *reinterpret_cast<uint16_t*>(at + 8 * c * P) = static_cast<uint16_t>(w[c]);
          *reinterpret_cast<uint16_t*>(at + (8 * c + 4) * P) = static_cast<uint16_t>(w[c] >> 16);
        }
      }
    }
    if (group_lane) pdst[r * groups + (16 * t >> gshift)] = par;
  }
  if (full) {
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < row_bytes; i += D)  // 16 rows' bytes / 16
      reinterpret_cast<uint4*>(gcodes)[i] = reinterpret_cast<const uint4*>(codes)[i];
    for (uint32_t i = threadIdx.x; i < 4 * groups; i += D)
      reinterpret_cast<uint4*>(gparams)[i] = reinterpret_cast<const uint4*>(params)[i];
  }
}

template <int D, typename TOut, bool ROT>
__global__ void __launch_bounds__(D) dequantize_ragged_kernel(const RaggedArgs a) {
  constexpr int U = D / 16;
  pdl_wait();
  pdl_trigger();
  const int4 e = load_entry(a, blockIdx.x);
  if (e.w == 0) return;
  const int h = blockIdx.y;
  const bool is_v = blockIdx.z != 0;
  const int b = is_v ? a.c.bits_v : a.c.bits_k, gshift = is_v ? a.c.gshift_v : a.c.gshift_k;
  const uint32_t t = threadIdx.x % U;  // thread of the row
  const int r = threadIdx.x / U;       // row of the tile
  const int first = e.y & 15;
  const bool valid = r >= first && r < first + e.w;
  const size_t row0 =
      (static_cast<size_t>(e.x) * a.c.kv_heads + h) * a.c.block_tokens + (e.y & ~15);
  const uint32_t row_bytes = D * b >> 3, groups = D >> gshift;
  const int e1 = b == 2 ? 7 : b == 4 ? 3 : 1;  // E - 1
  const int shift = b * (2 * t & e1);
  const uint32_t levels = (1u << b) - 1;
  float x[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = 0.0f;
  if (valid) {
    const float2 par =
        unpack_half2((is_v ? a.c.v_params : a.c.k_params)[(row0 + r) * groups + (16 * t >> gshift)]);
    uint32_t w[4];  // elements 2c, 2c + 1 in the halves
    if (!is_v) {
      const uint8_t* row = a.c.k_codes + (row0 + r) * row_bytes + 4 * (t * b >> 3);
#pragma unroll
      for (int c = 0; c < 4; ++c)
        w[c] = *reinterpret_cast<const uint32_t*>(row + c * (row_bytes >> 2));
    } else {
      const int P = 1 << v_piece_shift(D, b);
      const uint8_t* at = a.c.v_codes + row0 * row_bytes + v_half_offset(D, b, r, 2 * t);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t lo = *reinterpret_cast<const uint16_t*>(at + 8 * c * P);
        const uint32_t hi = *reinterpret_cast<const uint16_t*>(at + (8 * c + 4) * P);
        w[c] = lo | (hi << 16);
      }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // unit i / 2, half i mod 2
        const uint32_t q = (w[c] >> (shift + (i >> 1) * b + 16 * (i & 1))) & levels;
        // the code as binary32: its bits in the mantissa of 2^23
        const float code = __uint_as_float(q | 0x4b000000u) - 8388608.0f;
        x[(i >> 1) * 8 + 2 * c + (i & 1)] = fmaf(code, par.x, par.y);
      }
    }
  }
  if (ROT && !is_v) {  // k^ = H (H k^) / D
    rotate_row<D>(x, t);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] *= 1.0f / D;
  }
  if (valid) {
    TOut* dst = static_cast<TOut*>(const_cast<void*>(is_v ? a.v : a.k)) +
                static_cast<int64_t>(e.z + r - first) * (is_v ? a.v_stride : a.k_stride) + h * D +
                16 * t;
    store8<TOut>(dst, *reinterpret_cast<float(*)[8]>(x));
    store8<TOut>(dst + 8, *reinterpret_cast<float(*)[8]>(x + 8));
  }
}

template <int D, typename T>
cudaError_t launch_typed(const RaggedArgs& a, bool append, cudaStream_t stream) {
  const dim3 grid(a.num_entries, a.c.kv_heads, 2), block(D);
  const bool rot = a.c.rotate_keys;
  if (append)
    return rot ? launch_pdl(append_ragged_kernel<D, T, true>, grid, block, 0, stream, a)
               : launch_pdl(append_ragged_kernel<D, T, false>, grid, block, 0, stream, a);
  return rot ? launch_pdl(dequantize_ragged_kernel<D, T, true>, grid, block, 0, stream, a)
             : launch_pdl(dequantize_ragged_kernel<D, T, false>, grid, block, 0, stream, a);
}

template <int D>
cudaError_t launch_any(const RaggedArgs& a, bool append, cudaStream_t stream) {
  if (a.dtype == KVQ_F32) return launch_typed<D, float>(a, append, stream);
  if (a.dtype == KVQ_BF16) return launch_typed<D, __nv_bfloat16>(a, append, stream);
  return launch_typed<D, __half>(a, append, stream);
}

}  // namespace

cudaError_t launch_append_ragged(const RaggedArgs& a, cudaStream_t stream) {
  return a.c.head_dim == 128 ? launch_any<128>(a, true, stream) : launch_any<64>(a, true, stream);
}

cudaError_t launch_dequantize_ragged(const RaggedArgs& a, cudaStream_t stream) {
  return a.c.head_dim == 128 ? launch_any<128>(a, false, stream) : launch_any<64>(a, false, stream);
}

}  // namespace kvq
