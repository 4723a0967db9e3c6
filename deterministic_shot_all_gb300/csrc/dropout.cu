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

#include "activation.cuh"
#include "arx_internal.h"
#include "arx_rows.cuh"
#include "ops_launch.h"

namespace arx {
namespace {

constexpr int kTileThreads = 256;

// Tile of a block: 2^log_tx column groups by 256 >> log_tx rows.
struct Tile {
  uint32_t log_tx;
  __device__ __forceinline__ uint32_t group() const {
    return (blockIdx.x << log_tx) + (threadIdx.x & ((1u << log_tx) - 1u));
  }
  __device__ __forceinline__ uint32_t ty() const { return threadIdx.x >> log_tx; }
  __device__ __forceinline__ uint32_t rows() const { return kTileThreads >> log_tx; }
};

// The 8 columns of a group, or the first n of them where the row ends inside
// the group.  kVec: aligned vector accesses of whole groups.
template <int D, bool kVec>
struct Group {
  using S = typename Elem<D>::S;
  Pack<D, kVec ? 8 : 1> w[kVec ? 1 : 8];
  __device__ __forceinline__ void load(const S* p, int n) {
    if constexpr (kVec) {
      w[0].load(p);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < n)
          w[k].load(p + k);
        else
          w[k].zero();
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int k = 0; k < (kVec ? 1 : 8); ++k) w[k].zero();
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    if constexpr (kVec) {
      w[0].get(f);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = Elem<D>::widen(w[k].w);
    }
  }
  static __device__ __forceinline__ void put(S* p, const float (&f)[8], int n) {
    if constexpr (kVec) {
      Pack<D, 8> o;
      o.set(f);
      o.store(p);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < n) p[k] = Elem<D>::round(f[k]);
    }
  }
};

__device__ __forceinline__ void load_group_params(const void* p, int dtype, uint32_t c, int n, float (&f)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] = k < n ? load_param(p, dtype, c + k) : 0.0f;
}

template <int D, bool kVec>
__global__ void __launch_bounds__(kTileThreads) dropout_add_kernel(const arx_dropout_add_args a, Tile t,
                                                                   uint32_t threshold, float scale) {
  using S = typename Elem<D>::S;
  dependent_launch_prologue();
  const uint32_t g = t.group(), c = g * 8u;
  if (c >= a.cols) return;
  const int n = int(a.cols - c < 8 ? a.cols - c : 8);
  DropoutState d{};
  if (threshold) d = load_dropout(a.rng, threshold, scale);
  float b[8] = {};
  if (a.bias) load_group_params(a.bias, a.wdtype, c, n, b);
  const S* x = static_cast<const S*>(a.x) + c;
  const S* r = static_cast<const S*>(a.residual) + c;
  S* out = static_cast<S*>(a.out) + c;
  for (size_t row = size_t(blockIdx.y) * t.rows() + t.ty(); row < a.rows; row += size_t(gridDim.y) * t.rows()) {
    Group<D, kVec> vx, vr;
    vx.load(x + row * a.ldx, n);
    if (a.residual) vr.load(r + row * a.ldresidual, n);
    float f[8], h[8];
    vx.get(f);
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] += b[k];
    if (threshold) dropout8(f, d, g, uint32_t(row));
    if (a.residual) {
      vr.get(h);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] += h[k];
    }
    Group<D, kVec>::put(out + row * a.ldout, f, n);
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

template <int D, bool kVec>
__global__ void __launch_bounds__(kTileThreads) dropout_add_bwd_kernel(const arx_dropout_add_bwd_args a, Tile t,
                                                                       uint32_t threshold, float scale) {
  using S = typename Elem<D>::S;
  dependent_launch_prologue();
  const uint32_t g = t.group(), c = g * 8u;
  const int n = c >= a.cols ? 0 : int(a.cols - c < 8 ? a.cols - c : 8);
  DropoutState d{};
  if (threshold) d = load_dropout(a.rng, threshold, scale);
  float acc[8] = {};
  if (n > 0) {
    const S* dout = static_cast<const S*>(a.dout) + c;
    S* dx = static_cast<S*>(a.dx) + c;
    for (size_t row = size_t(blockIdx.y) * t.rows() + t.ty(); row < a.rows; row += size_t(gridDim.y) * t.rows()) {
      Group<D, kVec> v;
      v.load(dout + row * a.lddout, n);
      float f[8];
      v.get(f);
      if (threshold) dropout8(f, d, g, uint32_t(row));
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] += f[k];
      if (a.dx) Group<D, kVec>::put(dx + row * a.lddx, f, n);
    }
  }
  if (a.dbias) store_part(acc, t, c, a.cols, static_cast<float*>(a.workspace));
}

template <int D, bool kVec>
__global__ void __launch_bounds__(kTileThreads) act_grad_kernel(const ActGradCall a, Tile t) {
  using S = typename Elem<D>::S;
  dependent_launch_prologue();
  const uint32_t c = t.group() * 8u;
  const int n = c >= a.cols ? 0 : int(a.cols - c < 8 ? a.cols - c : 8);
  float acc[8] = {};
  if (n > 0) {
    const S* dout = static_cast<const S*>(a.dout) + c;
    const S* z = static_cast<const S*>(a.z) + c;
    S* dz = static_cast<S*>(a.dz) + c;
    for (size_t row = size_t(blockIdx.y) * t.rows() + t.ty(); row < a.rows; row += size_t(gridDim.y) * t.rows()) {
      Group<D, kVec> v, vz;
      v.load(dout + row * a.lddout, n);
      if (a.z) vz.load(z + row * a.ldz, n);
      float f[8], h[8];
      v.get(f);
      if (a.z) {
        vz.get(h);
        multiply_activation_grad<8>(f, h, a.act);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] += f[k];
      if (a.dz) Group<D, kVec>::put(dz + row * a.lddz, f, n);
    }
  }
  if (a.dbias) store_part(acc, t, c, a.cols, a.part);
}

// out[c] = sum over i < parts of p[i][c]: 32 columns per block, 8 lanes of
// partial rows added in order and then joined in order.
__global__ void __launch_bounds__(256) column_sum_kernel(const float* p0, void* out0, const float* p1, void* out1,
                                                         unsigned parts, uint64_t cols, int dtype) {
  __shared__ float join[8][32];
  dependent_launch_prologue();
  const float* p = blockIdx.y ? p1 : p0;
  void* out = blockIdx.y ? out1 : out0;
  if (!out) return;
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const size_t c = size_t(blockIdx.x) * 32 + tx;
  float s = 0.0f;
  if (c < cols)
    for (unsigned i = ty; i < parts; i += 8) s += p[size_t(i) * cols + c];
  join[ty][tx] = s;
  __syncthreads();
  if (ty == 0 && c < cols) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += join[i][tx];
    store_param(out, dtype, c, s);
  }
}

// Tile width of a matrix: as many groups as it has, up to 32.
Tile tile_of(uint64_t cols) {
  const uint64_t groups = (cols + 7) / 8;
  Tile t{0};
  while (t.log_tx < 5 && (uint64_t(1) << t.log_tx) < groups) ++t.log_tx;
  return t;
}

// Row chunks of the tiled kernels: about eight blocks of 256 threads for
// each of the 152 SMs over the whole grid, and no chunk without rows.
unsigned row_chunks(uint64_t rows, uint64_t cols) {
  const Tile t = tile_of(cols);
  const uint64_t groups = (cols + 7) / 8;
  const uint64_t tiles = (groups + (uint64_t(1) << t.log_tx) - 1) >> t.log_tx;
  const uint64_t per = kTileThreads >> t.log_tx;
  uint64_t chunks = 1216 / tiles;
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

template <int D>
cudaError_t dropout_add(const arx_dropout_add_args& a, bool vec, cudaStream_t st) {
  uint32_t T;
  float s;
  dropout_constants(a.p, &T, &s);
  auto k = vec ? dropout_add_kernel<D, true> : dropout_add_kernel<D, false>;
  return launch_op(k, tile_grid(a.rows, a.cols), kTileThreads, 0, st, a, tile_of(a.cols), T, s);
}

template <int D>
cudaError_t dropout_add_bwd(const arx_dropout_add_bwd_args& a, bool vec, cudaStream_t st) {
  uint32_t T;
  float s;
  dropout_constants(a.p, &T, &s);
  auto k = vec ? dropout_add_bwd_kernel<D, true> : dropout_add_bwd_kernel<D, false>;
  return launch_op(k, tile_grid(a.rows, a.cols), kTileThreads, 0, st, a, tile_of(a.cols), T, s);
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
    auto k = c.dtype == ARX_BF16 ? (vec ? act_grad_kernel<ARX_BF16, true> : act_grad_kernel<ARX_BF16, false>)
                                 : (vec ? act_grad_kernel<ARX_F16, true> : act_grad_kernel<ARX_F16, false>);
    const cudaError_t e = launch_op(k, tile_grid(c.rows, c.cols), kTileThreads, 0, st, c, tile_of(c.cols));
    if (e != cudaSuccess) return e;
  }
  return launch_column_sum(c.part, parts, c.cols, c.dbias, nullptr, nullptr, c.wdtype, st);
}

cudaError_t launch_column_sum(const float* p0, unsigned parts, uint64_t cols, void* out0, const float* p1,
                              void* out1, int dtype, cudaStream_t st) {
  if ((!out0 && !out1) || cols == 0) return cudaSuccess;
  return launch_op(column_sum_kernel, dim3(unsigned((cols + 31) / 32), out1 ? 2 : 1), 256, 0, st, p0, out0, p1, out1,
                   parts, cols, dtype);
}

}  // namespace arx
