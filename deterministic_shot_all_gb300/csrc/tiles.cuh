// Elementwise kernels that walk down a matrix in tiles of column groups and sum
// its columns on the way: tiles, access to rows of any alignment, partial sums
// (dropout.cu, gated_grad.cu).
#pragma once

#include <cuda_runtime.h>

#include <type_traits>

#include "arx_rows.cuh"
#include "ops_launch.h"

namespace arx {
namespace {

constexpr int kTileThreads = 256;
constexpr int kTileBlocks = 3;  // to an SM

// Tile of a block: 2^log_tx column groups by 256 >> log_tx rows.
struct Tile {
  uint32_t log_tx;
  __device__ __forceinline__ uint32_t group() const {
    return (blockIdx.x << log_tx) + (threadIdx.x & ((1u << log_tx) - 1u));
  }
  __device__ __forceinline__ uint32_t ty() const { return threadIdx.x >> log_tx; }
  __device__ __forceinline__ uint32_t rows() const { return kTileThreads >> log_tx; }
};

// How a thread gets the 8 columns of its group:
//  kVector  one aligned access of the whole group;
//  kStaged  rows off that alignment, 32 groups to a warp: the warp loads its 256
//           columns a line at a time, and exchanges them through shared memory;
//  kSingle  narrow matrices off that alignment: element by element.
enum Access { kVector, kStaged, kSingle };

// Rows that a thread has in flight at once, within 85 registers.
template <int D, int kAccess>
constexpr int kRowsOf = kAccess == kVector ? (D == ARX_F32 ? 2 : 4) : kAccess == kStaged ? 2 : 1;

template <int D, int kAccess>
struct Group {
  using S = typename Elem<D>::S;
  static constexpr int kStageBytes = kAccess == kStaged ? 256 * int(sizeof(S)) : 0;  // of a warp
  Pack<D, kAccess == kVector ? 8 : 1> w[kAccess == kVector ? 1 : 8];

  // p: the row's element at the group's first column (kStaged: at the warp's
  // first); n: the columns from there that exist, up to 8 (kStaged: any number).
  __device__ __forceinline__ void load(const S* p, int n) {
    if constexpr (kAccess == kVector) {
      w[0].load(p);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = kAccess == kStaged ? 32 * k + int(threadIdx.x & 31) : k;
        if (i < n)
          w[k].load(p + i);
        else
          w[k].zero();
      }
    }
  }
  __device__ __forceinline__ void get(float (&f)[8], S* stage) const {
    if constexpr (kAccess == kVector) {
      w[0].get(f);
    } else if constexpr (kAccess == kStaged) {
      const int lane = threadIdx.x & 31;
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 8; ++k) stage[32 * k + lane] = w[k].w;
      __syncwarp();
      const uint4* q = reinterpret_cast<const uint4*>(stage + 8 * lane);
      Pack<D, 8> v;
      const uint4 a = q[0];
      if constexpr (D == ARX_F32) {
        const uint4 b = q[1];
        v.w[0] = __uint_as_float(a.x), v.w[1] = __uint_as_float(a.y), v.w[2] = __uint_as_float(a.z),
        v.w[3] = __uint_as_float(a.w), v.w[4] = __uint_as_float(b.x), v.w[5] = __uint_as_float(b.y),
        v.w[6] = __uint_as_float(b.z), v.w[7] = __uint_as_float(b.w);
      } else {
        v.w[0] = a.x, v.w[1] = a.y, v.w[2] = a.z, v.w[3] = a.w;
      }
      v.get(f);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = Elem<D>::widen(w[k].w);
    }
  }
  static __device__ __forceinline__ void put(S* p, const float (&f)[8], int n, S* stage) {
    if constexpr (kAccess == kVector) {
      Pack<D, 8> o;
      o.set(f);
      o.store(p);
    } else if constexpr (kAccess == kStaged) {
      const int lane = threadIdx.x & 31;
      Pack<D, 8> o;
      o.set(f);
      __syncwarp();
      uint4* q = reinterpret_cast<uint4*>(stage + 8 * lane);
      if constexpr (D == ARX_F32) {
        q[0] = make_uint4(__float_as_uint(o.w[0]), __float_as_uint(o.w[1]), __float_as_uint(o.w[2]),
                          __float_as_uint(o.w[3]));
        q[1] = make_uint4(__float_as_uint(o.w[4]), __float_as_uint(o.w[5]), __float_as_uint(o.w[6]),
                          __float_as_uint(o.w[7]));
      } else {
        q[0] = make_uint4(o.w[0], o.w[1], o.w[2], o.w[3]);
      }
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (32 * k + lane < n) p[32 * k + lane] = stage[32 * k + lane];
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < n) p[k] = Elem<D>::round(f[k]);
    }
  }
};

// A thread's columns: its group, the group's first column, and what the
// accesses start from.
template <int D, int kAccess>
struct Columns {
  uint32_t group, first;  // generator group, its first column
  uint32_t at;            // column the accesses start from
  int n;                  // columns from there that exist (at most 8 unless staged)
  bool any;               // the thread takes part (all of a staged warp, or none)
  __device__ __forceinline__ Columns(const Tile& t, uint64_t cols) {
    group = t.group();
    first = group * 8u;
    at = kAccess == kStaged ? first - 8u * (threadIdx.x & 31) : first;
    any = at < cols;
    n = any ? (kAccess != kStaged && cols - at > 8 ? 8 : int(cols - at)) : 0;
  }
};

__device__ __forceinline__ void load_group_params(const void* p, int dtype, uint32_t c, uint64_t cols, float (&f)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] = c + k < cols ? load_param(p, dtype, c + k) : 0.0f;
}

// Joins the block's column sums over its row lanes, in order, and stores them
// as part[blockIdx.y][col].
__device__ __forceinline__ void store_part(const float (&acc)[8], const Tile& t, uint32_t c, uint64_t cols,
                                           float* part) {
  __shared__ float join[kTileThreads * 8];
  const uint32_t tx = threadIdx.x & ((1u << t.log_tx) - 1u);
  const uint32_t width = 8u << t.log_tx;
#pragma unroll
  for (int k = 0; k < 8; ++k) join[t.ty() * width + k * (1u << t.log_tx) + tx] = acc[k];
  __syncthreads();
  const uint32_t first = c - 8u * tx;
  for (uint32_t i = threadIdx.x; i < width; i += kTileThreads) {
    // Column i of the tile: element i % 8 of group i / 8.
    const uint32_t at = (i & 7u) * (1u << t.log_tx) + (i >> 3);
    float s = join[at];
    for (uint32_t y = 1; y < t.rows(); ++y) s += join[y * width + at];
    if (first + i < cols) part[size_t(blockIdx.y) * cols + first + i] = s;
  }
}

// Tile width of a matrix: as many groups as it has, up to 32.
inline Tile tile_of(uint64_t cols) {
  const uint64_t groups = (cols + 7) / 8;
  Tile t{0};
  while (t.log_tx < 5 && (uint64_t(1) << t.log_tx) < groups) ++t.log_tx;
  return t;
}

// Row chunks of the tiled kernels: as many blocks as 152 SMs hold at once over
// the whole grid, and no chunk without rows.
inline unsigned row_chunks(uint64_t rows, uint64_t cols) {
  const Tile t = tile_of(cols);
  const uint64_t groups = (cols + 7) / 8;
  const uint64_t tiles = (groups + (uint64_t(1) << t.log_tx) - 1) >> t.log_tx;
  const uint64_t per = kTileThreads >> t.log_tx;
  uint64_t chunks = 152 * kTileBlocks / tiles;
  if (chunks < 1) chunks = 1;
  const uint64_t most = (rows + per - 1) / per;
  if (chunks > most) chunks = most;
  return unsigned(chunks);
}

inline dim3 tile_grid(uint64_t rows, uint64_t cols) {
  const Tile t = tile_of(cols);
  const uint64_t groups = (cols + 7) / 8;
  return dim3(unsigned((groups + (uint64_t(1) << t.log_tx) - 1) >> t.log_tx), row_chunks(rows, cols));
}

// Calls f with the access of a matrix as a constant.
template <typename F>
cudaError_t with_access(bool vec, uint64_t cols, F f) {
  if (vec) return f(std::integral_constant<int, kVector>{});
  if (tile_of(cols).log_tx == 5) return f(std::integral_constant<int, kStaged>{});
  return f(std::integral_constant<int, kSingle>{});
}

}  // namespace
}  // namespace arx
