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
#include "tiles.cuh"

namespace arx {
namespace {

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
// partial rows, each added in order and then joined in order.  kBatch: loads of a
// lane in flight, ten for the 304 parts of two blocks to an SM at once.  Up to 128
// parts, four loads, the plain loop (28 parts behind [8192, 4096] of dropout's backward
// pass: 30.7 us in all, with ten 31.1).
constexpr unsigned kSumLanes = 32, kSumBatch = 10, kFewParts = 4 * kSumLanes;
template <unsigned kBatch>
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
    if constexpr (kBatch == 1) {
#pragma unroll 4
      for (unsigned i = ty; i < parts; i += kSumLanes) s += p[size_t(i) * cols + c];
    } else {
      for (unsigned i0 = ty; i0 < parts; i0 += kBatch * kSumLanes) {
        float v[kBatch];
#pragma unroll
        for (unsigned k = 0; k < kBatch; ++k)
          if (i0 + k * kSumLanes < parts) v[k] = p[size_t(i0 + k * kSumLanes) * cols + c];
#pragma unroll
        for (unsigned k = 0; k < kBatch; ++k)
          if (i0 + k * kSumLanes < parts) s += v[k];
      }
    }
  }
  join[ty][tx] = s;
  __syncthreads();
  // Warp ty joins column ty's lanes.
  s = warp_sum(join[tx][ty]);
  const size_t mine = size_t(blockIdx.x) * 32 + ty;
  if (tx == 0 && mine < cols) store_param(out, dtype, mine, s);
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
  const auto kernel = parts <= kFewParts ? column_sum_kernel<1> : column_sum_kernel<kSumBatch>;
  return launch_op(kernel, dim3(unsigned((cols + 31) / 32), out1 ? 2 : 1), 32 * kSumLanes, 0, st, p0, out0, p1, out1,
                   parts, cols, dtype);
}

}  // namespace arx
