// Copies of 16-bit matrices onto rows of 16 bytes, for products whose operands
// the copy engine cannot address (odd row lengths, views).
//
// Bound by memory: a row is read and written once, 128 consecutive bytes to an
// access of a warp.  The destination's words are the source's, or (a row on an
// odd element) joined from the halves of two neighbours, the second one from
// the next lane: loads of single elements would bring 18 bytes a cycle into an
// SM.  17.9 MB take 6 us.  16 words to a lane in flight, blocks of four warps:
// 8 words took 2 us more at 25 MB; blocks of eight warps 7 us less at 134 MB and
// 0.6 us more at 1 MB.
#include <cuda_runtime.h>

#include <cstdint>

#include "arx_device.cuh"
#include "arx_rows.cuh"
#include "ops_launch.h"
#include "spans.h"

namespace arx {
namespace {

constexpr uint32_t kWarps = 4, kWords = kRealignWords, kChunk = kRealignChunk;

// A warp's chunk of a row, from element c0 on.  kInside: every word that it
// looks at lies inside the row (with checks of each, issue slots bound the
// kernel: the product of 128 rows with [2047, 4099] took 24.0 us, so 20.0).
template <bool kInside>
__device__ __forceinline__ void realign_chunk(const Realign& a, const uint16_t* src, uint16_t* to, int64_t c0, bool odd,
                                              uint32_t lane) {
  const int64_t rest = a.cols - c0;
  const uint32_t* words = reinterpret_cast<const uint32_t*>(src - odd) + lane;
  // Word 32 i of the lane's: elements 2 (lane + 32 i) - odd and the next.
  // Elements outside the row are not touched.
  const auto load = [&](uint32_t i) -> uint32_t {
    if (kInside) return words[32 * i];
    if (64 * int64_t(i) > rest) return 0;  // the whole warp
    const int64_t c = realign_element(lane, i, odd);
    if (realign_both(c, c0, rest)) return words[32 * i];
    if (realign_lower(c, c0, rest)) return src[c];
    if (realign_upper(c, c0)) return uint32_t(src[0]) << 16;
    return 0;
  };
  uint32_t w[kWords + 1];
#pragma unroll
  for (uint32_t i = 0; i < kWords; ++i) w[i] = load(i);
  w[kWords] = odd && lane == 0 ? load(kWords) : 0;
  uint32_t* dst = reinterpret_cast<uint32_t*>(to) + lane;
  if (odd) {
#pragma unroll
    for (uint32_t i = 0; i < kWords; ++i) {
      const uint32_t up = __shfl_down_sync(0xFFFFFFFFu, w[i], 1), wrap = __shfl_sync(0xFFFFFFFFu, w[i + 1], 0);
      w[i] = __funnelshift_r(w[i], lane == 31 ? wrap : up, 16);
    }
  }
#pragma unroll
  for (uint32_t i = 0; i < kWords; ++i)
    if (kInside || 2 * int64_t(lane + 32 * i) < rest) dst[32 * i] = w[i];  // a last odd column's neighbour is padding
}

__global__ void __launch_bounds__(32 * kWarps) realign_kernel(const __grid_constant__ RealignSet set) {
  dependent_launch_prologue();
  const Realign& a = set.m[blockIdx.z];
  const uint32_t lane = threadIdx.x & 31;
  for (int64_t c0 = int64_t(blockIdx.x) * kChunk; c0 < a.cols; c0 += int64_t(gridDim.x) * kChunk)
    for (uint64_t row = blockIdx.y * kWarps + threadIdx.x / 32; row < a.rows; row += uint64_t(gridDim.y) * kWarps) {
      const uint16_t* src = a.src + row * a.ld + c0;
      uint16_t* to = a.dst + row * a.ld_dst + c0;
      const bool odd = reinterpret_cast<uintptr_t>(src) & 2;
      if (realign_inside(c0, a.cols, odd))
        realign_chunk<true>(a, src, to, c0, odd, lane);
      else
        realign_chunk<false>(a, src, to, c0, odd, lane);
    }
}

}  // namespace

cudaError_t launch_realign(const RealignSet& set, cudaStream_t st) {
  uint64_t rows = 0, cols = 0;
  for (int i = 0; i < set.n; ++i) {
    if (set.m[i].rows > rows) rows = set.m[i].rows;
    if (uint64_t(set.m[i].cols) > cols) cols = uint64_t(set.m[i].cols);
  }
  const uint64_t y = (rows + kWarps - 1) / kWarps, x = (cols + kChunk - 1) / kChunk;
  return launch_op(realign_kernel, dim3(unsigned(x), unsigned(y < 65535 ? y : 65535), unsigned(set.n)), 32 * kWarps, 0,
                   st, set);
}

}  // namespace arx
