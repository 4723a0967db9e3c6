// Layer norm, forward and backward.
//
// Bound by HBM: the forward reads x and writes y once, the backward reads dy
// and x (and dresidual) and writes dx once.  A row stays in its threads'
// registers between the pass that sums it and the pass that uses the sums.
#include <cuda_runtime.h>

#include "arx_internal.h"
#include "norm.cuh"
#include "ops_launch.h"

namespace arx {
namespace {

template <int D, int TPR, int RPC, int NV, int V>
__global__ void __launch_bounds__(TPR* RPC) norm_fwd_kernel(const arx_layer_norm_args a) {
  using S = typename Elem<D>::S;
  __shared__ float buf[RPC][2 * (TPR / 32)];
  dependent_launch_prologue();
  const size_t row = size_t(blockIdx.x) * RPC + threadIdx.x / TPR;
  if (RPC > 1 && row >= a.rows) return;  // whole warps; RPC > 1 has one warp per row and no barrier
  const S* x = static_cast<const S*>(a.x) + row * a.ldx;
  const uint32_t cols = uint32_t(a.cols);
  Pack<D, V> raw[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const uint32_t c = row_col<TPR, V>(i);
    if (c < cols)
      raw[i].load(x + c);
    else
      raw[i].zero();
  }
  float f[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) raw[i].get(f[i]);
  norm_row<D, TPR, NV, V>(f, cols, a.eps, a.weight, a.bias, a.wdtype, static_cast<S*>(a.y) + row * a.ldy,
                          a.mean ? a.mean + row : nullptr, a.rstd ? a.rstd + row : nullptr,
                          buf[threadIdx.x / TPR]);
}

// Any row length: one block per row, three passes over the row (the second
// and third mostly from cache).
template <int D>
__global__ void __launch_bounds__(512) norm_fwd_long_kernel(const arx_layer_norm_args a) {
  using S = typename Elem<D>::S;
  __shared__ float buf[2][16];
  dependent_launch_prologue();
  const size_t row = blockIdx.x;
  const S* x = static_cast<const S*>(a.x) + row * a.ldx;
  S* y = static_cast<S*>(a.y) + row * a.ldy;
  float s = 0.0f;
  for (size_t c = threadIdx.x; c < a.cols; c += 512) s += Elem<D>::widen(x[c]);
  const float mean = row_sum<512>(s, buf[0]) / float(a.cols);
  float q = 0.0f;
  for (size_t c = threadIdx.x; c < a.cols; c += 512) {
    const float d = Elem<D>::widen(x[c]) - mean;
    q += d * d;
  }
  const float rstd = 1.0f / sqrtf(row_sum<512>(q, buf[1]) / float(a.cols) + a.eps);
  for (size_t c = threadIdx.x; c < a.cols; c += 512) {
    float o = (Elem<D>::widen(x[c]) - mean) * rstd;
    if (a.weight) o *= load_param(a.weight, a.wdtype, c);
    if (a.bias) o += load_param(a.bias, a.wdtype, c);
    y[c] = Elem<D>::round(o);
  }
  if (threadIdx.x == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
}

// ---- backward -------------------------------------------------------------------

// Sums of two values over the row's threads (one barrier for both).
template <int TPR>
__device__ __forceinline__ void row_sum2(float& a, float& b, float* buf) {
  constexpr int kWarps = TPR / 32;
  a = warp_sum(a);
  b = warp_sum(b);
  if constexpr (TPR > 32) {
    if ((threadIdx.x & 31) == 0) {
      buf[(threadIdx.x % TPR) / 32] = a;
      buf[kWarps + (threadIdx.x % TPR) / 32] = b;
    }
    __syncthreads();
    a = buf[0];
    b = buf[kWarps];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) a += buf[i], b += buf[kWarps + i];
  }
}

template <int D, int NV, int V>
struct BwdRow {
  Pack<D, V> x[NV], dy[NV], dr[NV];
  float mean, rstd;
};

template <int D, int TPR, int NV, int V>
__device__ __forceinline__ void load_bwd_row(BwdRow<D, NV, V>& r, const arx_layer_norm_bwd_args& a, size_t row) {
  using S = typename Elem<D>::S;
  const S* x = static_cast<const S*>(a.x) + row * a.ldx;
  const S* dy = static_cast<const S*>(a.dy) + row * a.lddy;
  const S* dr = a.dresidual && a.dx ? static_cast<const S*>(a.dresidual) + row * a.lddresidual : nullptr;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const uint32_t c = row_col<TPR, V>(i);
    const bool in = c < uint32_t(a.cols);
    if (in) {
      r.x[i].load(x + c);
      r.dy[i].load(dy + c);
    }
    if (in && dr)
      r.dr[i].load(dr + c);
    else
      r.dr[i].zero();
  }
  r.mean = a.mean[row];
  r.rstd = a.rstd[row];
}

// Persistent: block b takes rows b, b + G, ... (RPC at a time) and keeps its
// columns' sums of dy * xh and dy in registers; they go to the workspace once,
// as part[0 or 1][b][cols], and column_sum_kernel adds the blocks in order.
// The next row's loads are in flight while a row is reduced.
template <int D, int TPR, int RPC, int NV, int V>
__global__ void __launch_bounds__(TPR* RPC) norm_bwd_kernel(const arx_layer_norm_bwd_args a) {
  using S = typename Elem<D>::S;
  constexpr int kWarps = TPR / 32;
  __shared__ float buf[2][RPC][2 * kWarps];
  extern __shared__ float join[];  // RPC > 1: [RPC][cols]
  dependent_launch_prologue();
  const uint32_t cols = uint32_t(a.cols);
  const int sub = threadIdx.x / TPR;
  const size_t step = size_t(gridDim.x) * RPC;
  float g[NV][V], acc_w[NV][V], acc_b[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const uint32_t c = row_col<TPR, V>(i);
#pragma unroll
    for (int k = 0; k < V; ++k) g[i][k] = 1.0f, acc_w[i][k] = 0.0f, acc_b[i][k] = 0.0f;
    if (a.weight && c < cols) load_params<V>(a.weight, a.wdtype, c, g[i]);
  }
  BwdRow<D, NV, V> cur, next;
  size_t row = size_t(blockIdx.x) * RPC + sub;
  if (row < a.rows) load_bwd_row<D, TPR, NV, V>(cur, a, row);
  int parity = 0;
  for (; row < a.rows; row += step) {
    if (row + step < a.rows) load_bwd_row<D, TPR, NV, V>(next, a, row + step);
    float xh[NV][V], q[NV][V], s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (row_col<TPR, V>(i) < cols) {
        cur.x[i].get(xh[i]);
        cur.dy[i].get(q[i]);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          xh[i][k] = (xh[i][k] - cur.mean) * cur.rstd;
          acc_w[i][k] += q[i][k] * xh[i][k];
          acc_b[i][k] += q[i][k];
          q[i][k] *= g[i][k];
          s1 += q[i][k];
          s2 += q[i][k] * xh[i][k];
        }
      }
    }
    if (a.dx) {
      row_sum2<TPR>(s1, s2, buf[parity][sub]);
      parity ^= 1;
      const float m1 = s1 / float(cols), m2 = s2 / float(cols);
      S* dx = static_cast<S*>(a.dx) + row * a.lddx;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const uint32_t c = row_col<TPR, V>(i);
        if (c >= cols) continue;
        float o[V];
        cur.dr[i].get(o);
#pragma unroll
        for (int k = 0; k < V; ++k) o[k] += cur.rstd * (q[i][k] - m1 - xh[i][k] * m2);
        Pack<D, V> out;
        out.set(o);
        out.store(dx + c);
      }
    }
    cur = next;
  }
  if (!a.dweight && !a.dbias) return;
  float* part = static_cast<float*>(a.workspace);
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if (which == 0 ? !a.dweight : !a.dbias) continue;
    float* to = part + (size_t(which) * gridDim.x + blockIdx.x) * cols;
    if constexpr (RPC > 1) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const uint32_t c = row_col<TPR, V>(i);
#pragma unroll
        for (int k = 0; k < V; ++k)
          if (c + k < cols) join[sub * cols + c + k] = which == 0 ? acc_w[i][k] : acc_b[i][k];
      }
      __syncthreads();
      for (uint32_t c = threadIdx.x; c < cols; c += TPR * RPC) {
        float s = join[c];
#pragma unroll
        for (int r = 1; r < RPC; ++r) s += join[r * cols + c];
        to[c] = s;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const uint32_t c = row_col<TPR, V>(i);
#pragma unroll
        for (int k = 0; k < V; ++k)
          if (c < cols) to[c + k] = which == 0 ? acc_w[i][k] : acc_b[i][k];
      }
    }
  }
}

// Any row length: dx with three passes over the row, and the column sums by
// norm_bwd_columns_kernel.
template <int D>
__global__ void __launch_bounds__(512) norm_bwd_long_kernel(const arx_layer_norm_bwd_args a) {
  using S = typename Elem<D>::S;
  __shared__ float buf[32];
  dependent_launch_prologue();
  const size_t row = blockIdx.x;
  const S* x = static_cast<const S*>(a.x) + row * a.ldx;
  const S* dy = static_cast<const S*>(a.dy) + row * a.lddy;
  const S* dr = a.dresidual ? static_cast<const S*>(a.dresidual) + row * a.lddresidual : nullptr;
  S* dx = static_cast<S*>(a.dx) + row * a.lddx;
  const float mean = a.mean[row], rstd = a.rstd[row];
  float s1 = 0.0f, s2 = 0.0f;
  for (size_t c = threadIdx.x; c < a.cols; c += 512) {
    float q = Elem<D>::widen(dy[c]);
    if (a.weight) q *= load_param(a.weight, a.wdtype, c);
    s1 += q;
    s2 += q * ((Elem<D>::widen(x[c]) - mean) * rstd);
  }
  row_sum2<512>(s1, s2, buf);
  const float m1 = s1 / float(a.cols), m2 = s2 / float(a.cols);
  for (size_t c = threadIdx.x; c < a.cols; c += 512) {
    float q = Elem<D>::widen(dy[c]);
    if (a.weight) q *= load_param(a.weight, a.wdtype, c);
    const float xh = (Elem<D>::widen(x[c]) - mean) * rstd;
    const float o = rstd * (q - m1 - xh * m2);
    dx[c] = Elem<D>::round(dr ? o + Elem<D>::widen(dr[c]) : o);
  }
}

// part[which][blockIdx.y][col] over the rows of chunk blockIdx.y.
template <int D>
__global__ void __launch_bounds__(256) norm_bwd_columns_kernel(const arx_layer_norm_bwd_args a) {
  using S = typename Elem<D>::S;
  __shared__ float join[2][8][32];
  dependent_launch_prologue();
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const size_t c = size_t(blockIdx.x) * 32 + tx;
  float sw = 0.0f, sb = 0.0f;
  if (c < a.cols)
    for (size_t row = size_t(blockIdx.y) * 8 + ty; row < a.rows; row += size_t(gridDim.y) * 8) {
      const float d = Elem<D>::widen(static_cast<const S*>(a.dy)[row * a.lddy + c]);
      const float xh = (Elem<D>::widen(static_cast<const S*>(a.x)[row * a.ldx + c]) - a.mean[row]) * a.rstd[row];
      sw += d * xh;
      sb += d;
    }
  join[0][ty][tx] = sw;
  join[1][ty][tx] = sb;
  __syncthreads();
  if (ty < 2 && c < a.cols) {
    float s = join[ty][0][tx];
#pragma unroll
    for (int i = 1; i < 8; ++i) s += join[ty][i][tx];
    static_cast<float*>(a.workspace)[(size_t(ty) * gridDim.y + blockIdx.y) * a.cols + c] = s;
  }
}

template <int D, int TPR, int RPC, int NV, int V>
cudaError_t fwd(const arx_layer_norm_args& a, cudaStream_t st) {
  return launch_op(norm_fwd_kernel<D, TPR, RPC, NV, V>, dim3(unsigned((a.rows + RPC - 1) / RPC)), TPR * RPC, 0, st, a);
}

template <int D>
cudaError_t fwd_any(const arx_layer_norm_args& a, bool vec, cudaStream_t st) {
  const uint64_t n = a.cols;
  if (vec) {
    if (n <= 256) return fwd<D, 32, 8, 1, 8>(a, st);
    if (n <= 512) return fwd<D, 32, 8, 2, 8>(a, st);
    if (n <= 1024) return fwd<D, 128, 1, 1, 8>(a, st);
    if (n <= 2048) return fwd<D, 256, 1, 1, 8>(a, st);
    if (n <= 4096) return fwd<D, 512, 1, 1, 8>(a, st);
    if (n <= 8192) return fwd<D, 512, 1, 2, 8>(a, st);
    if (n <= 16384) return fwd<D, 1024, 1, 2, 8>(a, st);
  } else {
    if (n <= 256) return fwd<D, 32, 8, 8, 1>(a, st);
    if (n <= 2048) return fwd<D, 256, 1, 8, 1>(a, st);
    if (n <= 4096) return fwd<D, 512, 1, 8, 1>(a, st);
    if (n <= 8192) return fwd<D, 512, 1, 16, 1>(a, st);
    if (n <= 16384) return fwd<D, 1024, 1, 16, 1>(a, st);
  }
  return launch_op(norm_fwd_long_kernel<D>, dim3(unsigned(a.rows)), 512, 0, st, a);
}

// Blocks of the persistent backward kernel: two of 512 threads on each of the
// 152 SMs, a constant so that the order of the sums depends on the sizes alone.
constexpr unsigned kBwdBlocks = 304;
// Row chunks of the column-sum kernel for long rows.
constexpr unsigned kColumnChunks = 64;

template <int D, int TPR, int RPC, int NV, int V>
cudaError_t bwd(const arx_layer_norm_bwd_args& a, unsigned* parts, cudaStream_t st) {
  const uint64_t need = (a.rows + RPC - 1) / RPC;
  const unsigned blocks = unsigned(need < kBwdBlocks ? need : kBwdBlocks);
  *parts = blocks;
  return launch_op(norm_bwd_kernel<D, TPR, RPC, NV, V>, dim3(blocks), TPR * RPC,
                   RPC > 1 ? size_t(RPC) * a.cols * 4 : 0, st, a);
}

template <int D>
cudaError_t bwd_any(const arx_layer_norm_bwd_args& a, bool vec, unsigned* parts, cudaStream_t st) {
  const uint64_t n = a.cols;
  if (vec) {
    if (n <= 256) return bwd<D, 32, 8, 1, 8>(a, parts, st);
    if (n <= 512) return bwd<D, 32, 8, 2, 8>(a, parts, st);
    if (n <= 1024) return bwd<D, 128, 1, 1, 8>(a, parts, st);
    if (n <= 2048) return bwd<D, 256, 1, 1, 8>(a, parts, st);
    if (n <= 4096) return bwd<D, 512, 1, 1, 8>(a, parts, st);
    if (n <= 8192) return bwd<D, 512, 1, 2, 8>(a, parts, st);
  } else {
    if (n <= 256) return bwd<D, 32, 8, 8, 1>(a, parts, st);
    if (n <= 2048) return bwd<D, 256, 1, 8, 1>(a, parts, st);
    if (n <= 4096) return bwd<D, 512, 1, 8, 1>(a, parts, st);
    if (n <= 8192) return bwd<D, 512, 1, 16, 1>(a, parts, st);
  }
  // The column sums first: dx may be written over dy or x.
  *parts = 0;
  if (a.dweight || a.dbias) {
    const uint64_t need = (a.rows + 7) / 8;
    *parts = unsigned(need < kColumnChunks ? need : kColumnChunks);
    const cudaError_t e = launch_op(norm_bwd_columns_kernel<D>, dim3(unsigned((a.cols + 31) / 32), *parts), 256, 0,
                                    st, a);
    if (e != cudaSuccess) return e;
  }
  if (!a.dx) return cudaSuccess;
  return launch_op(norm_bwd_long_kernel<D>, dim3(unsigned(a.rows)), 512, 0, st, a);
}

}  // namespace

size_t norm_bwd_parts(uint64_t rows, uint64_t cols) {
  (void)cols;
  return size_t(rows < kBwdBlocks ? rows : kBwdBlocks);
}

cudaError_t launch_layer_norm(const arx_layer_norm_args& a, bool vec, cudaStream_t st) {
  if (a.dtype == ARX_BF16) return fwd_any<ARX_BF16>(a, vec, st);
  if (a.dtype == ARX_F16) return fwd_any<ARX_F16>(a, vec, st);
  return fwd_any<ARX_F32>(a, vec, st);
}

cudaError_t launch_layer_norm_bwd(const arx_layer_norm_bwd_args& a, bool vec, cudaStream_t st) {
  unsigned parts = 0;
  cudaError_t e = cudaSuccess;
  if (a.rows > 0) {
    e = a.dtype == ARX_BF16  ? bwd_any<ARX_BF16>(a, vec, &parts, st)
        : a.dtype == ARX_F16 ? bwd_any<ARX_F16>(a, vec, &parts, st)
                             : bwd_any<ARX_F32>(a, vec, &parts, st);
    if (e != cudaSuccess) return e;
  }
  const float* p = static_cast<const float*>(a.workspace);
  return launch_column_sum(p, parts, a.cols, a.dweight, p + size_t(parts) * a.cols, a.dbias, a.wdtype, st);
}

}  // namespace arx
