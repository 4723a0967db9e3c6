// Dropout with bias and residual, the activation gradient of the matrix
// product's backward pass, and sums over rows.
//
// Bound by HBM, elementwise: a thread takes the 8 columns of one generator
// group (one Philox evaluation, about 80 integer instructions, for 8
// elements) of several rows.  Blocks tile the matrix by 32 groups (or fewer,
// for narrow matrices) and walk down a chunk of rows, so that a block's
// column sums stay in registers.
#include <cuda_runtime.h>

#include <cmath>
#include <type_traits>

#include "activation.cuh"
#include "arx_internal.h"
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

template <int D, int kAccess>
__global__ void __launch_bounds__(kTileThreads, kTileBlocks) dropout_add_kernel(const arx_dropout_add_args a, Tile t,
                                                                   uint32_t threshold, float scale) {
  constexpr int kRows = kRowsOf<D, kAccess>;
  using G = Group<D, kAccess>;
  using S = typename Elem<D>::S;
  __shared__ __align__(16) uint8_t stages[kTileThreads / 32 * G::kStageBytes + 16];
  S* stage = reinterpret_cast<S*>(stages + threadIdx.x / 32 * G::kStageBytes);
  dependent_launch_prologue();
  const Columns<D, kAccess> c(t, a.cols);
  if (!c.any) return;
  DropoutState d{};
  if (threshold) d = load_dropout(a.rng, threshold, scale);
  float b[8] = {};
  if (a.bias) load_group_params(a.bias, a.wdtype, c.first, a.cols, b);
  const S* x = static_cast<const S*>(a.x) + c.at;
  const S* r = static_cast<const S*>(a.residual) + c.at;
  S* out = static_cast<S*>(a.out) + c.at;
  const size_t step = size_t(gridDim.y) * t.rows();
  for (size_t row0 = size_t(blockIdx.y) * t.rows() + t.ty(); row0 < a.rows; row0 += kRows * step) {
    G vx[kRows], vr[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const size_t row = row0 + i * step;
      if (row >= a.rows) break;
      vx[i].load(x + row * a.ldx, c.n);
      if (a.residual) vr[i].load(r + row * a.ldresidual, c.n);
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const size_t row = row0 + i * step;
      if (row >= a.rows) break;
      uint4 random{};  // needs none of the loads in flight
      if (threshold) random = dropout_random(d, c.group, uint32_t(row));
      float f[8], h[8];
      vx[i].get(f, stage);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] += b[k];
      if (threshold) dropout_apply(f, d, random);
      if (a.residual) {
        vr[i].get(h, stage);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] += h[k];
      }
      G::put(out + row * a.ldout, f, c.n, stage);
    }
  }
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

template <int D, int kAccess>
__global__ void __launch_bounds__(kTileThreads, kTileBlocks) dropout_add_bwd_kernel(const arx_dropout_add_bwd_args a, Tile t,
                                                                       uint32_t threshold, float scale) {
  constexpr int kRows = kRowsOf<D, kAccess>;
  using G = Group<D, kAccess>;
  using S = typename Elem<D>::S;
  __shared__ __align__(16) uint8_t stages[kTileThreads / 32 * G::kStageBytes + 16];
  S* stage = reinterpret_cast<S*>(stages + threadIdx.x / 32 * G::kStageBytes);
  dependent_launch_prologue();
  const Columns<D, kAccess> c(t, a.cols);
  DropoutState d{};
  if (threshold) d = load_dropout(a.rng, threshold, scale);
  float acc[8] = {};
  if (c.any) {
    const S* dout = static_cast<const S*>(a.dout) + c.at;
    S* dx = static_cast<S*>(a.dx) + c.at;
    const size_t step = size_t(gridDim.y) * t.rows();
    for (size_t row0 = size_t(blockIdx.y) * t.rows() + t.ty(); row0 < a.rows; row0 += kRows * step) {
      G v[kRows];
  #pragma unroll
      for (int i = 0; i < kRows; ++i)
        if (row0 + i * step < a.rows) v[i].load(dout + (row0 + i * step) * a.lddout, c.n);
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        if (row0 + i * step >= a.rows) break;
        uint4 random{};  // needs none of the loads in flight
        if (threshold) random = dropout_random(d, c.group, uint32_t(row0 + i * step));
        float f[8];
        v[i].get(f, stage);
        if (threshold) dropout_apply(f, d, random);
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] += f[k];
        if (a.dx) G::put(dx + (row0 + i * step) * a.lddx, f, c.n, stage);
      }
    }
  }
  if (a.dbias) store_part(acc, t, c.first, a.cols, static_cast<float*>(a.workspace));
}

// dz = dout * act'(z), rounded to the operands' type where it is stored: the
// tensor cores take no other beside 16-bit weights and activations.  On dx and
// dw the rounding acts like a second one of their own (error against 64 bits
// 0.00234 in bf16, 0.00166 with dz in 32 bits); kept in two 16-bit parts, dz
// would double both products.  The column sums take it unrounded.
template <int D, int kAccess>
__global__ void __launch_bounds__(kTileThreads, kTileBlocks) act_grad_kernel(const ActGradCall a, Tile t) {
  constexpr int kRows = kRowsOf<D, kAccess>;
  using G = Group<D, kAccess>;
  using S = typename Elem<D>::S;
  __shared__ __align__(16) uint8_t stages[kTileThreads / 32 * G::kStageBytes + 16];
  S* stage = reinterpret_cast<S*>(stages + threadIdx.x / 32 * G::kStageBytes);
  dependent_launch_prologue();
  const Columns<D, kAccess> c(t, a.cols);
  float acc[8] = {};
  if (c.any) {
    const S* dout = static_cast<const S*>(a.dout) + c.at;
    const S* z = static_cast<const S*>(a.z) + c.at;
    S* dz = static_cast<S*>(a.dz) + c.at;
    const size_t step = size_t(gridDim.y) * t.rows();
    for (size_t row0 = size_t(blockIdx.y) * t.rows() + t.ty(); row0 < a.rows; row0 += kRows * step) {
      G v[kRows], vz[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const size_t row = row0 + i * step;
        if (row >= a.rows) break;
        v[i].load(dout + row * a.lddout, c.n);
        if (a.z) vz[i].load(z + row * a.ldz, c.n);
      }
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const size_t row = row0 + i * step;
        if (row >= a.rows) break;
        float f[8], h[8];
        v[i].get(f, stage);
        if (a.z) {
          vz[i].get(h, stage);
          multiply_activation_grad<8>(f, h, a.act);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] += f[k];
        if (a.dz) G::put(dz + row * a.lddz, f, c.n, stage);
      }
    }
  }
  if (a.dbias) store_part(acc, t, c.first, a.cols, a.part);
}

// out[c] = sum over i < parts of p[i][c]: 32 columns per block, 32 lanes of
// partial rows, each added in order and then joined in order.
constexpr unsigned kSumLanes = 32;
__global__ void __launch_bounds__(32 * kSumLanes) column_sum_kernel(const float* p0, void* out0, const float* p1,
                                                                    void* out1, unsigned parts, uint64_t cols,
                                                                    int dtype) {
  __shared__ float join[kSumLanes][33];
  dependent_launch_prologue();
  const float* p = blockIdx.y ? p1 : p0;
  void* out = blockIdx.y ? out1 : out0;
  if (!out) return;
  const unsigned tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const size_t c = size_t(blockIdx.x) * 32 + tx;
  float s = 0.0f;
  if (c < cols) {
#pragma unroll 4
    for (unsigned i = ty; i < parts; i += kSumLanes) s += p[size_t(i) * cols + c];
  }
  join[ty][tx] = s;
  __syncthreads();
  // Warp ty joins column ty's lanes.
  s = warp_sum(join[tx][ty]);
  const size_t mine = size_t(blockIdx.x) * 32 + ty;
  if (tx == 0 && mine < cols) store_param(out, dtype, mine, s);
}

// Tile width of a matrix: as many groups as it has, up to 32.
Tile tile_of(uint64_t cols) {
  const uint64_t groups = (cols + 7) / 8;
  Tile t{0};
  while (t.log_tx < 5 && (uint64_t(1) << t.log_tx) < groups) ++t.log_tx;
  return t;
}

// Row chunks of the tiled kernels: as many blocks as 152 SMs hold at once over
// the whole grid, and no chunk without rows.
unsigned row_chunks(uint64_t rows, uint64_t cols) {
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

dim3 tile_grid(uint64_t rows, uint64_t cols) {
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

template <int D>
cudaError_t dropout_add(const arx_dropout_add_args& a, bool vec, cudaStream_t st) {
  uint32_t T;
  float s;
  dropout_constants(a.p, &T, &s);
  return with_access(vec, a.cols, [&](auto m) {
    return launch_op(dropout_add_kernel<D, decltype(m)::value>, tile_grid(a.rows, a.cols), kTileThreads, 0, st, a,
                     tile_of(a.cols), T, s);
  });
}

template <int D>
cudaError_t dropout_add_bwd(const arx_dropout_add_bwd_args& a, bool vec, cudaStream_t st) {
  uint32_t T;
  float s;
  dropout_constants(a.p, &T, &s);
  return with_access(vec, a.cols, [&](auto m) {
    return launch_op(dropout_add_bwd_kernel<D, decltype(m)::value>, tile_grid(a.rows, a.cols), kTileThreads, 0, st, a,
                     tile_of(a.cols), T, s);
  });
}

template <int D>
cudaError_t act_grad(const ActGradCall& c, bool vec, cudaStream_t st) {
  return with_access(vec, c.cols, [&](auto m) {
    return launch_op(act_grad_kernel<D, decltype(m)::value>, tile_grid(c.rows, c.cols), kTileThreads, 0, st, c,
                     tile_of(c.cols));
  });
}

}  // namespace

size_t column_parts(uint64_t rows, uint64_t cols) { return rows && cols ? row_chunks(rows, cols) : 0; }

void dropout_constants(double p, uint32_t* threshold, float* scale) {
  // p in [0, 1] (checked by the caller); T = 65536 drops everything.
  const uint32_t T = uint32_t(std::nearbyint(p * 65536.0));
  *threshold = T;
  *scale = T >= 65536 ? 0.0f : float(65536.0 / (65536.0 - double(T)));
}

cudaError_t launch_dropout_add(const arx_dropout_add_args& a, bool vec, cudaStream_t st) {
  if (a.dtype == ARX_BF16) return dropout_add<ARX_BF16>(a, vec, st);
  if (a.dtype == ARX_F16) return dropout_add<ARX_F16>(a, vec, st);
  return dropout_add<ARX_F32>(a, vec, st);
}

cudaError_t launch_dropout_add_bwd(const arx_dropout_add_bwd_args& a, bool vec, cudaStream_t st) {
  unsigned parts = 0;
  if (a.rows > 0 && (a.dx || a.dbias)) {
    parts = row_chunks(a.rows, a.cols);
    const cudaError_t e = a.dtype == ARX_BF16  ? dropout_add_bwd<ARX_BF16>(a, vec, st)
                          : a.dtype == ARX_F16 ? dropout_add_bwd<ARX_F16>(a, vec, st)
                                               : dropout_add_bwd<ARX_F32>(a, vec, st);
    if (e != cudaSuccess) return e;
  }
  return launch_column_sum(static_cast<const float*>(a.workspace), parts, a.cols, a.dbias, nullptr, nullptr,
                           a.wdtype, st);
}

cudaError_t launch_act_grad(const ActGradCall& c, bool vec, cudaStream_t st) {
  unsigned parts = 0;
  if (c.rows > 0 && (c.dz || c.dbias)) {
    parts = row_chunks(c.rows, c.cols);
    const cudaError_t e = c.dtype == ARX_BF16 ? act_grad<ARX_BF16>(c, vec, st) : act_grad<ARX_F16>(c, vec, st);
    if (e != cudaSuccess) return e;
  }
  return launch_column_sum(c.part, parts, c.cols, c.dbias, nullptr, nullptr, c.wdtype, st);
}

cudaError_t launch_column_sum(const float* p0, unsigned parts, uint64_t cols, void* out0, const float* p1,
                              void* out1, int dtype, cudaStream_t st) {
  if ((!out0 && !out1) || cols == 0) return cudaSuccess;
  return launch_op(column_sum_kernel, dim3(unsigned((cols + 31) / 32), out1 ? 2 : 1), 32 * kSumLanes, 0, st, p0, out0, p1, out1,
                   parts, cols, dtype);
}

}  // namespace arx
