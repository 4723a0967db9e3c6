// Copies of 16-bit matrices onto rows of 16 bytes, for products whose operands
// the copy engine cannot address (odd row lengths, views).
//
// Bound by memory: a row is read and written once, 128 consecutive bytes to an
// access of a warp.  The destination's words are the source's, or (a row on an
// odd element) joined from the halves of two neighbours, the second one from
// the next lane: loads of single elements would bring 18 bytes a cycle into an
// SM.  About 2.3 us and 2.9 TB/s read (16.8 MB: 8.0 us); 16 words to a lane in
// flight and blocks of four warps: 4 words took 3 us more at 25 MB, 32 words 4.
#include <cuda_runtime.h>

#include <cstdint>

#include "arx_device.cuh"
#include "arx_rows.cuh"
#include "ops_launch.h"

namespace arx {
namespace {

constexpr uint32_t kWarps = 4, kWords = 16, kChunk = 64 * kWords;  // kWords words to a lane; elements to a warp

__global__ void __launch_bounds__(32 * kWarps) realign_kernel(const __grid_constant__ RealignPair pair) {
  dependent_launch_prologue();
  const Realign& a = pair.m[blockIdx.z];
  const uint32_t lane = threadIdx.x & 31;
  // An element's index in its row; signed, as the word before the first is looked at.
  for (int64_t chunk = blockIdx.x; chunk * int64_t(kChunk) < a.cols; chunk += gridDim.x)
    for (uint64_t row = blockIdx.y * kWarps + threadIdx.x / 32; row < a.rows; row += uint64_t(gridDim.y) * kWarps) {
      const uint16_t* src = a.src + row * a.ld;
      const int64_t cols = a.cols, c0 = chunk * int64_t(kChunk);
      const bool odd = reinterpret_cast<uintptr_t>(src + c0) & 2;
      // Word k of the chunk: elements c0 + 2 k - odd and the next.  Elements
      // outside the row are not touched.
      const auto load = [&](uint32_t k) -> uint32_t {
        const int64_t c = c0 + 2 * int64_t(k) - odd;
        if (c >= 0 && c + 1 < cols) return *reinterpret_cast<const uint32_t*>(src + c);
        if (c >= 0 && c < cols) return src[c];
        if (c == -1) return uint32_t(src[0]) << 16;
        return 0;
      };
      uint32_t w[kWords + 1];
#pragma unroll
      for (uint32_t i = 0; i < kWords; ++i) w[i] = load(lane + 32 * i);
      w[kWords] = odd && lane == 0 ? load(32 * kWords) : 0;
      uint32_t* dst = reinterpret_cast<uint32_t*>(a.dst + row * a.ld_dst + c0);
#pragma unroll
      for (uint32_t i = 0; i < kWords; ++i) {
        if (odd) {
          const uint32_t up = __shfl_down_sync(0xFFFFFFFFu, w[i], 1), wrap = __shfl_sync(0xFFFFFFFFu, w[i + 1], 0);
          w[i] = __funnelshift_r(w[i], lane == 31 ? wrap : up, 16);
        }
        const int64_t c = c0 + 2 * (lane + 32 * int64_t(i));
        if (c < cols) dst[lane + 32 * i] = w[i];  // a last odd column's neighbour is padding
      }
    }
}

}  // namespace

cudaError_t launch_realign(const RealignPair& pair, cudaStream_t st) {
  uint64_t rows = 0, cols = 0;
  for (int i = 0; i < pair.n; ++i) {
    if (pair.m[i].rows > rows) rows = pair.m[i].rows;
    if (uint64_t(pair.m[i].cols) > cols) cols = uint64_t(pair.m[i].cols);
  }
  const uint64_t y = (rows + kWarps - 1) / kWarps, x = (cols + kChunk - 1) / kChunk;
  return launch_op(realign_kernel, dim3(unsigned(x), unsigned(y < 65535 ? y : 65535), unsigned(pair.n)), 32 * kWarps, 0,
                   st, pair);
}

}  // namespace arx
