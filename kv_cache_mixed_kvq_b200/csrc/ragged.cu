// Ragged quantize-and-append and its read-back (kvq_quantize_append_ragged,
// kvq_dequantize_ragged): packed tokens of rows of any lengths, each 16-position
// tile that takes tokens named by one entry of the slot map.
//
// One CTA handles one entry of one kv head, keys or values.  A thread owns a
// unit of 8 consecutive elements of one token (one 16-byte load of a 16-bit
// type), the D/8 units of a row in consecutive lanes.  Bits and group sizes
// are runtime values (uniform over the launch): a unit's eight codes are built
// from the same binary32 steps as in quantize.cuh,
//   mn, mx = group min and max (xor-shuffles over the group's lanes);
//   scale = (mx - mn) / (2^b - 1);  inv = 1 / scale;
//   code = rint((x - mn) * inv), 0 for a degenerate group,
// and both layouts keep a unit's codes at one place of a word: element
// d = 8u + m (unit u, m = 0..7) sits at bit 16 (m mod 2) + b (u mod E) of
//   keys:   word u/E of slice m/2 of its row,
//   values: (position k of the tile) half k mod 2 of word (k/8) W + u/E of
//           lane 4m + (k mod 8)/2 (bit offset without the 16 (m mod 2)),
// E = 16/b, so a register per slice holds elements 2c and 2c+1 in its halves,
// shifted by b (u mod E), and an exclusive or over the E lanes of a word
// completes it (the fields are disjoint).
//
// Bound: HBM traffic for long chunks (2 D es bytes in, D (bk + bv) / 8 + 4
// (D/Gk + D/Gv) out per token and head), launch latency for single tokens.
// Whole tiles are assembled in shared memory and leave as 16-byte stores; an
// edge tile's words go to global memory one by one, so that positions of no
// entry keep their bytes.
#include "common.cuh"
#include "internal.h"
#include "serve.h"

namespace kvq {
namespace {

// Entry e of the map if it names places inside the cache and the packed
// tokens; count 0 (and an error flag) otherwise.
__device__ __forceinline__ int4 load_entry(const RaggedArgs& a, int e) {
  int4 m = __ldg(a.map + e);
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

// Walsh-Hadamard butterfly h = 1, 2, ..., D/2 of a row whose unit u is in
// lane u: stages below 8 inside the thread, the others by xor-shuffles.
template <int D>
__device__ __forceinline__ void rotate_units(float (&x)[8], int u) {
#pragma unroll
  for (int h = 1; h < 8; h *= 2)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((i & h) == 0) {
        const float p = x[i], q = x[i + h];
        x[i] = __fadd_rn(p, q);
        x[i + h] = __fsub_rn(p, q);
      }
#pragma unroll
  for (int m = 1; m < D / 8; m *= 2) {
    const bool upper = (u & m) != 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float y = __shfl_xor_sync(0xffffffffu, x[i], m);
      x[i] = upper ? __fsub_rn(y, x[i]) : __fadd_rn(x[i], y);
    }
  }
}

// Byte offset of a value word's half of element 8u + m, position k, in a tile.
__device__ __forceinline__ int v_half_offset(int D, int b, int k, int u, int m) {
  const int N = D * b / 16, P = min(16, N), W = D * b / 128;
  const int n = 4 * ((k / 8) * W + u * b / 16) + 2 * (k & 1);
  return (n / P) * 32 * P + (4 * m + (k & 7) / 2) * P + n % P;
}

template <int D, typename TIn, bool ROT>
__global__ void __launch_bounds__(2 * D) append_ragged_kernel(const RaggedArgs a) {
  constexpr int U = D / 8;
  __shared__ __align__(16) uint8_t codes[16 * D];  // a tile at 8 bits
  __shared__ __align__(16) uint32_t params[16 * (D / 32)];
  pdl_wait();
  pdl_trigger();
  const int4 e = load_entry(a, blockIdx.x);
  if (e.w == 0) return;
  const int h = blockIdx.y;
  const bool is_v = blockIdx.z != 0;
  const int b = is_v ? a.c.bits_v : a.c.bits_k, G = is_v ? a.c.group_v : a.c.group;
  const int u = threadIdx.x % U, r = threadIdx.x / U;  // unit, row of the tile
  const int first = e.y & 15;
  const bool full = e.w == 16;
  const bool valid = r >= first && r < first + e.w;
  const size_t row0 =
      (static_cast<size_t>(e.x) * a.c.kv_heads + h) * a.c.block_tokens + (e.y & ~15);

  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = 0.0f;
  if (valid) {
    const TIn* src = static_cast<const TIn*>(is_v ? a.v : a.k) +
                     static_cast<int64_t>(e.z + r - first) * (is_v ? a.v_stride : a.k_stride) +
                     h * D + 8 * u;
    Load8<TIn>::run(src, x);
  }
  if (ROT && !is_v) rotate_units<D>(x, u);

  float mn = x[0], mx = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    mn = fminf(mn, x[i]);
    mx = fmaxf(mx, x[i]);
  }
  for (int m = 1; m < G / 8; m <<= 1) {
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, m));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, m));
  }
  mn = (mn == 0.0f) ? 0.0f : mn;  // a zero extreme is stored as +0
  mx = (mx == 0.0f) ? 0.0f : mx;
  const int levels = (1 << b) - 1;
  const float scale = __fdiv_rn(__fsub_rn(mx, mn), static_cast<float>(levels));
  const float inv = __fdiv_rn(1.0f, scale);
  const bool flat = scale == 0.0f || !isfinite(scale) || !isfinite(inv);
  const float f = flat ? 0.0f : inv, z = flat ? 0.0f : mn;
  const int shift = b * (u & (16 / b - 1));
  uint32_t w[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int lo = __float2int_rn(__fmul_rn(__fsub_rn(x[2 * c], z), f)) & levels;
    const int hi = __float2int_rn(__fmul_rn(__fsub_rn(x[2 * c + 1], z), f)) & levels;
    w[c] = static_cast<uint32_t>(lo | (hi << 16)) << shift;
  }
  for (int m = 1; m < 16 / b; m <<= 1) {
#pragma unroll
    for (int c = 0; c < 4; ++c) w[c] |= __shfl_xor_sync(0xffffffffu, w[c], m);
  }

  // the word's first lane stores it; the group's first lane its parameters
  const bool word_lane = (u & (16 / b - 1)) == 0, group_lane = u % (G / 8) == 0;
  const uint32_t par = pack_half2(__float2half_rn(scale), __float2half_rn(mn));
  const int row_bytes = D * b / 8, groups = D / G;
  uint8_t* gcodes = is_v ? a.c.v_codes + row0 * row_bytes  // (a tile has 16 rows' bytes)
                         : a.c.k_codes + row0 * row_bytes;
  uint32_t* gparams = (is_v ? a.c.v_params : a.c.k_params) + row0 * groups;
  uint8_t* cdst = full ? codes : gcodes;
  uint32_t* pdst = full ? params : gparams;
  if (valid) {
    if (word_lane) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (!is_v) {
          *reinterpret_cast<uint32_t*>(cdst + r * row_bytes + c * (row_bytes / 4) +
                                       4 * (u * b / 16)) = w[c];
        } else {
          *reinterpret_cast<uint16_t*>(cdst + v_half_offset(D, b, r, u, 2 * c)) =
              static_cast<uint16_t>(w[c]);
          *reinterpret_cast<uint16_t*>(cdst + v_half_offset(D, b, r, u, 2 * c + 1)) =
              static_cast<uint16_t>(w[c] >> 16);
        }
      }
    }
    if (group_lane) pdst[r * groups + u / (G / 8)] = par;
  }
  if (full) {
    __syncthreads();
    for (int i = threadIdx.x; i < row_bytes; i += 2 * D)  // 16 rows' bytes / 16
      reinterpret_cast<uint4*>(gcodes)[i] = reinterpret_cast<const uint4*>(codes)[i];
    for (int i = threadIdx.x; i < 4 * groups; i += 2 * D)
      reinterpret_cast<uint4*>(gparams)[i] = reinterpret_cast<const uint4*>(params)[i];
  }
}

template <int D, typename TOut, bool ROT>
__global__ void __launch_bounds__(2 * D) dequantize_ragged_kernel(const RaggedArgs a) {
  constexpr int U = D / 8;
  pdl_wait();
  pdl_trigger();
  const int4 e = load_entry(a, blockIdx.x);
  if (e.w == 0) return;
  const int h = blockIdx.y;
  const bool is_v = blockIdx.z != 0;
  const int b = is_v ? a.c.bits_v : a.c.bits_k, G = is_v ? a.c.group_v : a.c.group;
  const int u = threadIdx.x % U, r = threadIdx.x / U;
  const int first = e.y & 15;
  const bool valid = r >= first && r < first + e.w;
  const size_t row0 =
      (static_cast<size_t>(e.x) * a.c.kv_heads + h) * a.c.block_tokens + (e.y & ~15);
  const int row_bytes = D * b / 8, groups = D / G;
  const int shift = b * (u & (16 / b - 1));
  const uint32_t levels = (1u << b) - 1;
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = 0.0f;
  if (valid) {
    const float2 par =
        unpack_half2((is_v ? a.c.v_params : a.c.k_params)[(row0 + r) * groups + u / (G / 8)]);
    uint32_t w[4];
    if (!is_v) {
      const uint8_t* row = a.c.k_codes + (row0 + r) * row_bytes + 4 * (u * b / 16);
#pragma unroll
      for (int c = 0; c < 4; ++c)
        w[c] = *reinterpret_cast<const uint32_t*>(row + c * (row_bytes / 4));
    } else {
      const uint8_t* tile = a.c.v_codes + row0 * row_bytes;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t lo =
            *reinterpret_cast<const uint16_t*>(tile + v_half_offset(D, b, r, u, 2 * c));
        const uint32_t hi =
            *reinterpret_cast<const uint16_t*>(tile + v_half_offset(D, b, r, u, 2 * c + 1));
        w[c] = lo | (hi << 16);
      }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      x[2 * c] = fmaf(static_cast<float>((w[c] >> shift) & levels), par.x, par.y);
      x[2 * c + 1] = fmaf(static_cast<float>((w[c] >> (16 + shift)) & levels), par.x, par.y);
    }
  }
  if (ROT && !is_v) {  // k^ = H (H k^) / D
    rotate_units<D>(x, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= 1.0f / D;
  }
  if (valid) {
    TOut* dst = static_cast<TOut*>(const_cast<void*>(is_v ? a.v : a.k)) +
                static_cast<int64_t>(e.z + r - first) * (is_v ? a.v_stride : a.k_stride) + h * D +
                8 * u;
    store8<TOut>(dst, x);
  }
}

template <int D, typename T>
cudaError_t launch_typed(const RaggedArgs& a, bool append, cudaStream_t stream) {
  const dim3 grid(a.num_entries, a.c.kv_heads, 2), block(2 * D);
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
