// Chunk attention: launches, and the kernel that joins the partial results of
// units of work cut by a border between two CTAs' shares.
#include <mutex>
#include <set>
#include <utility>

#include "chunk.cuh"

namespace kvq {
namespace {

// Rows of a unit that one CTA joins (4 warps, a row at a time each).
constexpr int kCombineRows = 16;

// A unit's pieces lie in place 1 of the CTA that began it and in place 0 of
// the CTAs after it, up to the one that ended it:
//   M = max m_i,  o = sum 2^(m_i - M) o_i / sum 2^(m_i - M) l_i.
// Bound: its few megabytes of traffic, mostly the launch.
template <int D>
__global__ void __launch_bounds__(128) combine_kernel(const ChunkArgs a, int grid) {
  constexpr int N = D / 32;  // elements per lane
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_trigger();
  // the header in two loads, both under way before either is looked at
  const int4* hd = reinterpret_cast<const int4*>(a.ws_head) + (blockIdx.x * 2 + 1) * 2;
  const int4 h0 = hd[0], h1 = hd[1];
  if (h0.x == 0 || h1.y != 0) return;
  const int start = h0.y, h = h0.z, row0 = h0.w, rows = h1.x;
  for (int i = warp; i < kCombineRows; i += 4) {
    const int r = blockIdx.y * kCombineRows + i;
    if (r >= rows) return;
    float o[N], m = -INFINITY, l = 0.0f;
    bool nothing = false;  // the row sees no position: its output is 0
#pragma unroll
    for (int k = 0; k < N; ++k) o[k] = 0.0f;
    int place = blockIdx.x * 2 + 1;
    for (int c = blockIdx.x; c < grid; ++c, place = 2 * c) {
      const size_t prow = static_cast<size_t>(place) * a.part_rows + r;
      const float2 ml = a.ws_ml[prow];
      nothing = ml.y < 0.0f;
      const float mm = fmaxf(m, ml.x), base = mm == -INFINITY ? 0.0f : mm;
      const float f = exp2_approx(m - base), g = exp2_approx(ml.x - base);
      l = l * f + ml.y * g;
      m = mm;
      const float* src = a.ws_o + prow * D + lane * N;
#pragma unroll
      for (int k = 0; k < N; ++k) o[k] = o[k] * f + src[k] * g;
      if (a.ws_head[place * 8 + 5] != 0) break;
    }
    const int br = row0 + r;
    const float inv = 1.0f / l;
    const size_t orow =
        (static_cast<size_t>(start + br / a.gq) * a.q_heads + h * a.gq + br % a.gq) * D + lane * N;
#pragma unroll
    for (int k = 0; k < N; ++k) store_out(a.out, a.out_dtype, orow + k, nothing ? 0.0f : o[k] * inv);
  }
}

// Opts the kernel in to its shared memory, once per device; refuses a library
// whose launches would not allocate the registers that the kernel's split counts
// on (the build checks the same, with a message).
cudaError_t prepare(const void* fn) {
  static std::mutex mu;
  static std::set<std::pair<int, const void*>> done;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  if (done.count({dev, fn})) return cudaSuccess;
  cudaFuncAttributes attr;
  e = cudaFuncGetAttributes(&attr, fn);
  if (e == cudaSuccess && (attr.numRegs + 7) / 8 * 8 != chunk::kRegsLaunch)
    e = cudaErrorInvalidConfiguration;
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, chunk::kSmemMax);
  if (e == cudaSuccess) done.insert({dev, fn});
  return e;
}

template <int D, int PIECES, int NT, bool ROT>
cudaError_t launch(const ChunkArgs& a, int grid, cudaStream_t stream) {
  auto* kernel = &chunk::chunk_kernel<chunk::Cfg<D, PIECES, NT>, ROT>;
  cudaError_t e = prepare(reinterpret_cast<const void*>(kernel));
  if (e != cudaSuccess) return e;
  e = launch_pdl(kernel, dim3(grid), dim3(chunk::kThreads), chunk::kSmemMax, stream, a);
  if (e != cudaSuccess || a.whole_units) return e;
  return launch_pdl(combine_kernel<D>, dim3(grid, (a.part_rows + kCombineRows - 1) / kCombineRows),
                    dim3(128), 0, stream, a, grid);
}

template <int D, int PIECES, int NT>
cudaError_t launch_rot(const ChunkArgs& a, int grid, cudaStream_t stream) {
  return a.c.rotate_keys ? launch<D, PIECES, NT, true>(a, grid, stream)
                         : launch<D, PIECES, NT, false>(a, grid, stream);
}

template <int D>
cudaError_t launch_d(const ChunkArgs& a, int pieces, int grid, cudaStream_t stream) {
  if (pieces == 1) {
    if (tile_tokens(1, D, a.c.bits_k + a.c.bits_v) == 128)
      return launch_rot<D, 1, 128>(a, grid, stream);
    if constexpr (D == 128) return launch_rot<D, 1, 64>(a, grid, stream);
  }
  if (pieces == 2) return launch<D, 2, 64, false>(a, grid, stream);
  return launch_rot<D, 3, 64>(a, grid, stream);
}

}  // namespace

cudaError_t launch_chunk(const ChunkArgs& a, int pieces, int grid, cudaStream_t stream) {
  return a.c.head_dim == 128 ? launch_d<128>(a, pieces, grid, stream)
                             : launch_d<64>(a, pieces, grid, stream);
}

}  // namespace kvq
