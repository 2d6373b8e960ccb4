// Attention of a chunk of new tokens over the packed cache
// (kvq_chunk_attention).
//
//   s_it = scale q_i . k^_t,  p_it = exp(s_it - m_i),  o_i = sum_t p_it v^_t / sum_t p_it
// in one pass over the positions t with a running maximum m_i and sum l_i:
// when the maximum grows from m to m', o_i and l_i are scaled by
// exp(m - m').  The query heads of one kv head share its keys, so a row of
// the tile is a (token, head) pair: row r of batch row b is token r / gq of
// its new ones, head r mod gq of the kv head.
//
// One CTA takes 16 rows of one kv head and goes through the positions 32 at a
// time, dequantized to binary32 in shared memory; a warp owns 4 rows, a lane
// one position (scores) or D/32 elements (output).
#include "common.cuh"
#include "internal.h"
#include "serve.h"

namespace kvq {
namespace {

constexpr int kRows = 16, kTile = 32, kThreads = 128, kPer = kRows / 4;

template <int D>
__global__ void __launch_bounds__(kThreads) chunk_kernel(const ChunkArgs a) {
  __shared__ float s_q[kRows][D];
  __shared__ float s_k[kTile][D + 1];
  __shared__ float s_v[kTile][D];
  pdl_wait();
  pdl_trigger();
  const int h = blockIdx.y, t = threadIdx.x, lane = t & 31, warp = t >> 5;
  // the batch row of this tile
  int tile = blockIdx.x, b = 0, start = 0, n = 0;
  for (; b < a.batch; ++b) {
    start = __ldg(a.cu + b);
    n = __ldg(a.cu + b + 1) - start;
    if (start < 0 || n < 0 || n > a.max_q_len || start > a.num_tokens - n) {
      if (t == 0 && h == 0) flag_error(a.err, KVQ_DEVERR_BAD_POS);
      n = 0;
    }
    const int tiles = (n * a.gq + kRows - 1) / kRows;
    if (tile < tiles) break;
    tile -= tiles;
  }
  if (b == a.batch) return;
  int len = __ldg(a.seq_lens + b);
  const int lim = min(a.max_seq_len, a.capacity);
  if (len > lim) {
    if (t == 0) flag_error(a.err, KVQ_DEVERR_SEQ_LEN);
    len = lim;
  }
  len = max(len, 0);
  const int rows = n * a.gq;

  for (int i = t; i < kRows * D; i += kThreads) {
    const int r = tile * kRows + i / D, d = i % D;
    float x = 0.0f;
    if (r < rows)
      x = load_elem(a.q, a.q_dtype,
                    static_cast<size_t>(start + r / a.gq) * a.q_stride +
                        (h * a.gq + r % a.gq) * D + d);
    s_q[i / D][d] = x;
  }
  __syncthreads();
  if (a.c.rotate_keys) {  // H q / D
    for (int hh = 1; hh < D; hh *= 2) {
      for (int i = t; i < kRows * D / 2; i += kThreads) {
        const int r = i / (D / 2), j = i % (D / 2), d = (j / hh) * 2 * hh + j % hh;
        const float x = s_q[r][d], y = s_q[r][d + hh];
        s_q[r][d] = x + y;
        s_q[r][d + hh] = x - y;
      }
      __syncthreads();
    }
    for (int i = t; i < kRows * D; i += kThreads) s_q[i / D][i % D] *= 1.0f / D;
    __syncthreads();
  }

  float m[kPer], l[kPer], o[kPer][D / 32];
  int limit[kPer];
  int last = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int r = tile * kRows + warp * kPer + i;
    m[i] = -INFINITY;
    l[i] = 0.0f;
    limit[i] = r < rows ? (a.causal ? min(len, max(0, len - n + r / a.gq + 1)) : len) : 0;
#pragma unroll
    for (int j = 0; j < D / 32; ++j) o[i][j] = 0.0f;
  }
  {
    const int r = min(rows, (tile + 1) * kRows) - 1;
    last = a.causal ? min(len, max(0, len - n + r / a.gq + 1)) : len;
  }
  const int bk = a.c.bits_k, bv = a.c.bits_v, ek = 16 / bk, ev = 16 / bv;
  for (int p0 = 0; p0 < last; p0 += kTile) {
    __syncthreads();
    for (int i = t; i < kTile * D; i += kThreads) {
      const int p = p0 + i / D, d = i % D, u = d / 8, mm = d % 8;
      float kx = 0.0f, vx = 0.0f;
      if (p < last) {
        int block = b, local = p;
        if (a.table != nullptr) {
          block = __ldg(a.table + static_cast<size_t>(b) * a.pages_per_seq + (p >> a.page_shift));
          local = p & ((1 << a.page_shift) - 1);
        }
        if (block < 0 || block >= a.c.blocks) {
          if (d == 0) flag_error(a.err, KVQ_DEVERR_BAD_PAGE);
        } else {
          const size_t row =
              (static_cast<size_t>(block) * a.c.kv_heads + h) * a.c.block_tokens + local;
          const uint32_t kw = *reinterpret_cast<const uint32_t*>(
              a.c.k_codes + row * (D * bk / 8) + (mm / 2) * (D * bk / 32) + 4 * (u / ek));
          const float2 kp = unpack_half2(a.c.k_params[row * (D / a.c.group) + d / a.c.group]);
          kx = fmaf(static_cast<float>((kw >> (16 * (mm & 1) + bk * (u % ek))) & ((1u << bk) - 1)),
                    kp.x, kp.y);
          const int k = local & 15, N = D * bv / 16, P = min(16, N), W = D * bv / 128;
          const int nn = 4 * ((k / 8) * W + u / ev);
          const uint32_t vw = *reinterpret_cast<const uint32_t*>(
              a.c.v_codes + (row - k) * (D * bv / 8) + (nn / P) * 32 * P +
              (4 * mm + (k & 7) / 2) * P + nn % P);
          const float2 vp = unpack_half2(a.c.v_params[row * (D / a.c.group_v) + d / a.c.group_v]);
          vx = fmaf(static_cast<float>((vw >> (16 * (k & 1) + bv * (u % ev))) & ((1u << bv) - 1)),
                    vp.x, vp.y);
        }
      }
      s_k[i / D][d] = kx;
      s_v[i / D][d] = vx;
    }
    __syncthreads();
    float s[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) s[i] = 0.0f;
    for (int d = 0; d < D; ++d) {
      const float kx = s_k[lane][d];
#pragma unroll
      for (int i = 0; i < kPer; ++i) s[i] = fmaf(s_q[warp * kPer + i][d], kx, s[i]);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      float x = p0 + lane < limit[i] ? s[i] * a.sm_scale_log2 : -INFINITY;
      float mx = x;
#pragma unroll
      for (int w = 16; w >= 1; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      const float mn = fmaxf(m[i], mx);
      const float base = mn == -INFINITY ? 0.0f : mn;  // (a row that sees nothing yet)
      const float keep = exp2f(m[i] - base);
      x = exp2f(x - base);
      s[i] = x;
#pragma unroll
      for (int w = 16; w >= 1; w >>= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
      l[i] = l[i] * keep + x;
      m[i] = mn;
#pragma unroll
      for (int j = 0; j < D / 32; ++j) o[i][j] *= keep;
    }
    for (int p = 0; p < kTile; ++p) {
      float vx[D / 32];
#pragma unroll
      for (int j = 0; j < D / 32; ++j) vx[j] = s_v[p][lane + 32 * j];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const float w = __shfl_sync(0xffffffffu, s[i], p);
#pragma unroll
        for (int j = 0; j < D / 32; ++j) o[i][j] = fmaf(w, vx[j], o[i][j]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int r = tile * kRows + warp * kPer + i;
    if (r >= rows) continue;
    const size_t row =
        (static_cast<size_t>(start + r / a.gq) * a.q_heads + h * a.gq + r % a.gq) * D;
    const float f = l[i] > 0.0f ? 1.0f / l[i] : 0.0f;
#pragma unroll
    for (int j = 0; j < D / 32; ++j)
      store_out(a.out, a.out_dtype, row + lane + 32 * j, o[i][j] * f);
  }
}

}  // namespace

cudaError_t launch_chunk(const ChunkArgs& a, cudaStream_t stream) {
  const long long tiles =
      (static_cast<long long>(a.num_tokens) * a.gq) / kRows + a.batch;
  const dim3 grid(static_cast<unsigned>(tiles), a.c.kv_heads);
  return a.c.head_dim == 128
             ? launch_pdl(chunk_kernel<128>, grid, dim3(kThreads), 0, stream, a)
             : launch_pdl(chunk_kernel<64>, grid, dim3(kThreads), 0, stream, a);
}

}  // namespace kvq
