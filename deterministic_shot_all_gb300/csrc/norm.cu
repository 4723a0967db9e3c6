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

constexpr unsigned kSms = 152;

template <int D, int TPR, int RPC, int NV, int V>
__global__ void __launch_bounds__(TPR* RPC) norm_fwd_kernel(const arx_layer_norm_args a, float inv_cols) {
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
  norm_row<D, TPR, NV, V>(f, cols, inv_cols, a.eps, a.weight, a.bias, a.wdtype, static_cast<S*>(a.y) + row * a.ldy,
                          a.mean ? a.mean + row : nullptr, a.rstd ? a.rstd + row : nullptr,
                          buf[threadIdx.x / TPR]);
}

// Many rows: persistent, as the backward kernel below, with the weights and
// biases in registers and rows coming in through a ring.  (One block to a row
// reads 8 bytes of 32-bit parameters for every 4 of a 16-bit row: 45.6 us at
// [8192, 4096], 2.3 times the bytes' time.)
template <int T, int RPC>
constexpr int kFwdBlocks = T * RPC >= 512 ? 1 : T * RPC > 256 ? 2 : 3;

template <int D, int T, int RPC, int NV, int V, int kRing>
__global__ void __launch_bounds__(T* RPC, kFwdBlocks<T, RPC>)
    norm_fwd_ring_kernel(const arx_layer_norm_args a, uint32_t slot, float inv_cols) {
  using S = typename Elem<D>::S;
  constexpr int kWarps = T / 32;
  __shared__ float buf[2][RPC][kWarps];
  extern __shared__ __align__(16) uint8_t smem[];  // [RPC][kRing][slot]
  dependent_launch_prologue();
  const uint32_t cols = uint32_t(a.cols), sub = threadIdx.x / T;
  uint8_t* ring = smem + sub * kRing * slot;
  const S* gx = static_cast<const S*>(a.x);
  const size_t step = size_t(gridDim.x) * RPC;
  size_t row = size_t(blockIdx.x) * RPC + sub;
  const auto start = [&](size_t r, uint32_t at) {  // one group, empty past the last row
    if (r < a.rows) copy_matrix_row<D, T, NV, V>(ring + at * slot, gx, a.ldx, r, a.rows, cols);
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i + 1 < kRing; ++i) start(row + i * step, i);
  float w[NV][V], b[NV][V];
  hold_params<T, NV, V>(w, a.weight, a.wdtype, cols, 1.0f);
  hold_params<T, NV, V>(b, a.bias, a.wdtype, cols, 0.0f);
  uint32_t at = 0;
  for (; row < a.rows; row += step) {
    cp_async_wait<kRing - 2>();
    if (V == 1) row_barrier<T, RPC>();
    const uint8_t* x = ring + at * slot + row_offset<V>(gx + row * a.ldx);
    float f[NV][V], s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t c = row_col<T, V>(i);
#pragma unroll
      for (int k = 0; k < V; ++k) f[i][k] = 0.0f;
      if (c < cols) read_shared<D, V>(x + c * sizeof(S), f[i]);
#pragma unroll
      for (int k = 0; k < V; ++k) s += f[i][k];
    }
    // The slot of the row before, which every thread has read.
    start(row + (kRing - 1) * step, at == 0 ? kRing - 1 : at - 1);
    const float mean = row_sum<T, RPC>(s, buf[0][sub]) * inv_cols;
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (row_col<T, V>(i) < cols)
#pragma unroll
        for (int k = 0; k < V; ++k) f[i][k] -= mean, q += f[i][k] * f[i][k];
    const float rstd = 1.0f / sqrtf(row_sum<T, RPC>(q, buf[1][sub]) * inv_cols + a.eps);
    S* y = static_cast<S*>(a.y) + row * a.ldy;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t c = row_col<T, V>(i);
      if (c >= cols) continue;
      float o[V];
#pragma unroll
      for (int k = 0; k < V; ++k) o[k] = f[i][k] * rstd * w[i][k] + b[i][k];
      Pack<D, V> out;
      out.set(o);
      out.store(y + c);
    }
    if (threadIdx.x % T == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    at = at + 1 == kRing ? 0 : at + 1;
  }
  cp_async_wait<0>();
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
  const float mean = row_sum<512, 1>(s, buf[0]) / float(a.cols);
  float q = 0.0f;
  for (size_t c = threadIdx.x; c < a.cols; c += 512) {
    const float d = Elem<D>::widen(x[c]) - mean;
    q += d * d;
  }
  const float rstd = 1.0f / sqrtf(row_sum<512, 1>(q, buf[1]) / float(a.cols) + a.eps);
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

// T threads to a row, RPC rows to a block, up to 16 columns to a thread (32 in
// the longest rows).  Persistent: the block's rows are RPC b, RPC (b + G), ...;
// it keeps the weights and its columns' sums of dy * xh and dy in registers,
// and the sums go to the workspace once, as part[0 or 1][b][cols], for
// column_sum_kernel to add the blocks in order.  Rows arrive through a ring of
// kRing rows in shared memory.
//
// [8192, 4096] bf16: 8 columns to a thread took 75 us, the issue slots going
// to the sums over 16 warps and each row's bookkeeping; 32 to a thread with the
// weights read anew for every row 88 us, waiting for them.
template <int T, int RPC>
constexpr int kBwdBlocks = T * RPC > 256 ? 1 : 2;

template <int D, int T, int RPC, int NV, int V, int kRing>
__global__ void __launch_bounds__(T* RPC, kBwdBlocks<T, RPC>) norm_bwd_kernel(const arx_layer_norm_bwd_args a,
                                                                           uint32_t slot, float inv_cols) {
  using S = typename Elem<D>::S;
  constexpr int kWarps = T / 32;
  constexpr bool kHold = NV * V <= 16 && T <= 512;  // the weights, xh and q stay in registers
  __shared__ float buf[2][RPC][2 * kWarps];
  extern __shared__ __align__(16) uint8_t smem[];  // [RPC][kRing][x, dy, dresidual][slot]
  dependent_launch_prologue();
  const uint32_t cols = uint32_t(a.cols);
  const bool res = a.dresidual && a.dx;
  const uint32_t arrays = res ? 3 : 2, sub = threadIdx.x / T;
  uint8_t* ring = smem + sub * kRing * arrays * slot;
  const S *gx = static_cast<const S*>(a.x), *gdy = static_cast<const S*>(a.dy),
          *gdr = static_cast<const S*>(a.dresidual);

  const auto start = [&](size_t row, uint32_t at) {  // one group, empty past the last row
    if (row < a.rows) {
      uint8_t* dst = ring + at * arrays * slot;
      copy_matrix_row<D, T, NV, V>(dst, gx, a.ldx, row, a.rows, cols);
      copy_matrix_row<D, T, NV, V>(dst + slot, gdy, a.lddy, row, a.rows, cols);
      if (res) copy_matrix_row<D, T, NV, V>(dst + 2 * slot, gdr, a.lddresidual, row, a.rows, cols);
    }
    cp_async_commit();
  };

  float acc_w[NV][V] = {}, acc_b[NV][V] = {}, w[kHold ? NV : 1][V];
  const size_t step = size_t(gridDim.x) * RPC;
  size_t row = size_t(blockIdx.x) * RPC + sub;
#pragma unroll
  for (int i = 0; i + 1 < kRing; ++i) start(row + i * step, i);
  if constexpr (kHold) hold_params<T, NV, V>(w, a.weight, a.wdtype, cols, 1.0f);
  float mean = 0.0f, rstd = 0.0f;
  if (row < a.rows) mean = a.mean[row], rstd = a.rstd[row];
  uint32_t at = 0;
  int parity = 0;
  for (; row < a.rows; row += step) {
    float next_mean = 0.0f, next_rstd = 0.0f;
    if (row + step < a.rows) next_mean = a.mean[row + step], next_rstd = a.rstd[row + step];
    cp_async_wait<kRing - 2>();
    if (V == 1) row_barrier<T, RPC>();
    // The slot of the row before, which every thread has read for the last time.
    start(row + (kRing - 1) * step, at == 0 ? kRing - 1 : at - 1);
    const uint8_t* base = ring + at * arrays * slot;
    const uint8_t* x = base + row_offset<V>(gx + row * a.ldx);
    const uint8_t* dy = base + slot + row_offset<V>(gdy + row * a.lddy);
    const uint8_t* dr = base + 2 * slot + row_offset<V>(gdr + row * a.lddresidual);
    float xh[kHold ? NV : 1][V], q[kHold ? NV : 1][V], sums[2] = {0.0f, 0.0f};
    // Unit i's xh and q = dy * weight; the first pass also adds up.
    const auto unit = [&](int i, uint32_t c, float (&h)[V], float (&p)[V], bool first) {
      read_shared<D, V>(x + c * sizeof(S), h);
      read_shared<D, V>(dy + c * sizeof(S), p);
      float g[V];
      if constexpr (!kHold) {
#pragma unroll
        for (int k = 0; k < V; ++k) g[k] = 1.0f;
        if (a.weight) load_params<V>(a.weight, a.wdtype, c, g);
      }
#pragma unroll
      for (int k = 0; k < V; ++k) {
        h[k] = (h[k] - mean) * rstd;
        if (first) {
          acc_w[i][k] += p[k] * h[k];
          acc_b[i][k] += p[k];
        }
        p[k] *= kHold ? w[kHold ? i : 0][k] : g[k];
        if (first) {
          sums[0] += p[k];
          sums[1] += p[k] * h[k];
        }
      }
    };
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t c = row_col<T, V>(i);
      if (c < cols) unit(i, c, xh[kHold ? i : 0], q[kHold ? i : 0], true);
    }
    if (a.dx) {
      row_sums<T, RPC, 2>(sums, buf[parity][sub]);
      parity ^= 1;
      const float m1 = sums[0] * inv_cols, m2 = sums[1] * inv_cols;
      S* dx = static_cast<S*>(a.dx) + row * a.lddx;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const uint32_t c = row_col<T, V>(i);
        if (c >= cols) continue;
        float (&h)[V] = xh[kHold ? i : 0], (&p)[V] = q[kHold ? i : 0], o[V];
        if constexpr (!kHold) unit(i, c, h, p, false);
#pragma unroll
        for (int k = 0; k < V; ++k) o[k] = 0.0f;
        if (res) read_shared<D, V>(dr + c * sizeof(S), o);
#pragma unroll
        for (int k = 0; k < V; ++k) o[k] += rstd * (p[k] - m1 - h[k] * m2);
        Pack<D, V> out;
        out.set(o);
        out.store(dx + c);
      }
    }
    mean = next_mean, rstd = next_rstd;
    at = at + 1 == kRing ? 0 : at + 1;
  }
  cp_async_wait<0>();
  if (!a.dweight && !a.dbias) return;
  float* part = static_cast<float*>(a.workspace);
  float* join = reinterpret_cast<float*>(smem);  // RPC > 1: [RPC][cols], once the rings are done with
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if (which == 0 ? !a.dweight : !a.dbias) continue;
    float* to = part + (size_t(which) * gridDim.x + blockIdx.x) * cols;
    if (RPC > 1) __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t c = row_col<T, V>(i);
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (c < cols) (RPC > 1 ? join + sub * cols : to)[c + k] = which == 0 ? acc_w[i][k] : acc_b[i][k];
    }
    if constexpr (RPC > 1) {
      __syncthreads();
      for (uint32_t c = threadIdx.x; c < cols; c += T * RPC) {
        float s = join[c];
#pragma unroll
        for (int r = 1; r < RPC; ++r) s += join[r * cols + c];
        to[c] = s;
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
  float sums[2] = {s1, s2};
  row_sums<512, 1, 2>(sums, buf);
  const float m1 = sums[0] / float(a.cols), m2 = sums[1] / float(a.cols);
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
  return launch_op(norm_fwd_kernel<D, TPR, RPC, NV, V>, dim3(unsigned((a.rows + RPC - 1) / RPC)), TPR * RPC, 0, st, a,
                   1.0f / float(a.cols));
}

// Shared memory of an SM that its blocks' rings may fill, and of one block.
constexpr size_t kRingBytes = 222 * 1024, kBlockRingBytes = 220 * 1024;

template <int D, int T, int RPC, int NV, int V>
cudaError_t fwd_ring(const arx_layer_norm_args& a, cudaStream_t st) {
  constexpr int kRing = 5;
  const uint32_t slot = row_slot(a.cols, sizeof(typename Elem<D>::S), V);
  const size_t smem = size_t(RPC) * kRing * slot;  // at most 5 x 32 KB, 8192 columns of fp32
  size_t per_sm = kRingBytes / (smem + 2048);
  if (per_sm > kFwdBlocks<T, RPC>) per_sm = kFwdBlocks<T, RPC>;
  const uint64_t need = (a.rows + RPC - 1) / RPC, most = per_sm * kSms;
  constexpr auto kernel = norm_fwd_ring_kernel<D, T, RPC, NV, V, kRing>;
  const cudaError_t e = allow_dynamic_smem<kernel>(kBlockRingBytes);
  if (e != cudaSuccess) return e;
  return launch_op(kernel, dim3(unsigned(need < most ? need : most)), T * RPC, smem, st, a, slot,
                   1.0f / float(a.cols));
}

// Does a forward pass go through the ring?  One block to a row, with more
// threads the fewer columns each has the sooner it ends, is the other form, and
// the better one up to four rows to an SM.  Above, the ring gains as it holds
// the parameters (the more their bytes beside the rows') and by the rows in
// flight; its few blocks cost where rows are short and many, or read element
// by element.  Measured, time of the ring by that of the other form, 609 to
// 16,384 rows (16-bit rows with 32-bit parameters; with 16-bit ones; 32-bit rows):
//   up to 256 columns   to 2,000 rows .61 to 1.0; 1.0 to 1.2; .64 to 1.0
//                       from 3,000    1.1 to 1.7; 1.25 to 1.7; 1.1 to 1.6
//   512  aligned        .74 to 1.0; .88 to 1.1; .75 to 1.2
//        off 16 bytes   .56 to 1.2; 1.1 to 2.1, from 8,192 rows .6 to .85; .6 to 1.2
//   1024 aligned        to 2,000 rows .8 to 1.3; .9 to 1.3; 1.1 to 1.4
//                       from 3,000    .7 to .9; .7 to 1.0; 1.1 to 1.2
//        off 16 bytes   .9 to 1.3; 1.1 to 1.85; 1.0 to 1.3
//   2048 aligned        .7 to .95; .75 to 1.1; .9 to 1.2
//        off 16 bytes   .9 to 1.2; 1.0 to 1.8; .95 to 1.3
//   4096 aligned        .6 to .95; .65 to 1.0; .85 to 1.05
//        off 16 bytes   .85 to 1.1; 1.1 to 1.5, from 4,000 rows .9 to 1.0; .85 to 1.1
//   above               .3 to .6; .3 to .9; .55 to .8
// In the ring 320 threads to rows of up to 5120 columns, against 512: .55 to .9
// of the time, 32-bit rows of whole units 1.0 to 1.1 at 5120 columns, .85 at 4200.
template <int D>
bool through_ring(const arx_layer_norm_args& a, bool vec) {
  const uint64_t n = a.cols;
  if (a.rows <= 4 * kSms) return false;
  const bool wide = (a.weight || a.bias) && a.wdtype == ARX_F32, more = a.rows > 16 * kSms;
  if (n <= 256) return wide && !more;
  if (n <= 512) return vec || wide || a.rows > 48 * kSms;
  if (n <= 1024) return vec && D != ARX_F32 && more;
  if (n <= 2048) return vec && D != ARX_F32;
  if (n <= 4096) return vec || wide || more;
  return true;
}

template <int D>
cudaError_t fwd_any(const arx_layer_norm_args& a, bool vec, cudaStream_t st) {
  const uint64_t n = a.cols;
  const bool ring = through_ring<D>(a, vec);
  constexpr bool kHalf = D != ARX_F32;
  if (vec) {
    if (n <= 256) return ring ? fwd_ring<D, 32, 8, 1, 8>(a, st) : fwd<D, 32, 4, 1, 8>(a, st);
    if (n <= 512) return ring ? fwd_ring<D, 32, 8, 2, 8>(a, st) : fwd<D, 32, 4, 2, 8>(a, st);
    if constexpr (kHalf) {
      if (n <= 1024 && ring) return fwd_ring<D, 64, 4, 2, 8>(a, st);
      if (n <= 2048 && ring) return fwd_ring<D, 128, 2, 2, 8>(a, st);
    }
    if (n <= 1024) return fwd<D, 128, 1, 1, 8>(a, st);
    if (n <= 2048) return fwd<D, 256, 1, 1, 8>(a, st);
    if (n <= 4096) return ring ? fwd_ring<D, 256, 1, 2, 8>(a, st) : fwd<D, 512, 1, 1, 8>(a, st);
    if (n <= 5120 && ring) return fwd_ring<D, 320, 1, 2, 8>(a, st);
    if (n <= 8192) return ring ? fwd_ring<D, 512, 1, 2, 8>(a, st) : fwd<D, 1024, 1, 1, 8>(a, st);
    if (n <= 16384) return fwd<D, 512, 1, 4, 8>(a, st);
  } else {
    if (n <= 256) return ring ? fwd_ring<D, 32, 8, 8, 1>(a, st) : fwd<D, 32, 4, 8, 1>(a, st);
    if (n <= 512) return ring ? fwd_ring<D, 32, 8, 16, 1>(a, st) : fwd<D, 128, 1, 8, 1>(a, st);
    if (n <= 1024) return fwd<D, 128, 1, 8, 1>(a, st);
    if (n <= 2048) return fwd<D, 256, 1, 8, 1>(a, st);
    if (n <= 4096) return ring ? fwd_ring<D, 256, 1, 16, 1>(a, st) : fwd<D, 512, 1, 8, 1>(a, st);
    if (n <= 5120 && ring) return fwd_ring<D, 320, 1, 16, 1>(a, st);
    if (n <= 8192) return ring ? fwd_ring<D, 512, 1, 16, 1>(a, st) : fwd<D, 1024, 1, 8, 1>(a, st);
    if (n <= 16384) return fwd<D, 1024, 1, 16, 1>(a, st);
  }
  return launch_op(norm_fwd_long_kernel<D>, dim3(unsigned(a.rows)), 512, 0, st, a);
}

// Row chunks of the column-sum kernel for long rows.
constexpr unsigned kColumnChunks = 64;
// As many blocks as 152 SMs hold at once: a constant, so that the order of the
// sums depends on the call alone: sizes, type, alignment, and whether dresidual (an
// array more in the ring) is there.
template <int D, int T, int RPC, int NV, int V, int kRing>
cudaError_t bwd_ring(const arx_layer_norm_bwd_args& a, unsigned* parts, uint32_t slot, size_t smem, cudaStream_t st) {
  size_t per_sm = kRingBytes / (smem + 2048);
  if (per_sm > kBwdBlocks<T, RPC>) per_sm = kBwdBlocks<T, RPC>;
  if (per_sm < 1) per_sm = 1;
  const uint64_t need = (a.rows + RPC - 1) / RPC;
  const unsigned blocks = unsigned(need < per_sm * kSms ? need : per_sm * kSms);
  *parts = blocks;
  constexpr auto kernel = norm_bwd_kernel<D, T, RPC, NV, V, kRing>;
  const cudaError_t e = allow_dynamic_smem<kernel>(kBlockRingBytes);
  if (e != cudaSuccess) return e;
  return launch_op(kernel, dim3(blocks), T * RPC, smem, st, a, slot, 1.0f / float(a.cols));
}

// Three rows in the ring, two where three are too large; *done is false where
// two are as well.
template <int D, int T, int RPC, int NV, int V>
cudaError_t bwd(const arx_layer_norm_bwd_args& a, unsigned* parts, bool* done, cudaStream_t st) {
  const size_t size = sizeof(typename Elem<D>::S);
  const uint32_t slot = row_slot(a.cols, size, V);
  const size_t row = size_t(a.dresidual && a.dx ? 3 : 2) * slot * RPC;
  // (Two rows of two arrays hold the RPC rows of sums, too.)
  *done = 2 * row <= kBlockRingBytes;
  if (!*done) return cudaSuccess;
  return 3 * row <= kBlockRingBytes ? bwd_ring<D, T, RPC, NV, V, 3>(a, parts, slot, 3 * row, st)
                                    : bwd_ring<D, T, RPC, NV, V, 2>(a, parts, slot, 2 * row, st);
}

// 320 threads to rows of 4097 to 5120 columns off 16 bytes, whose columns are
// read one by one (512 threads take up to 1.1 times as long); aligned ones gain
// nothing by it ([8192, 5120] with dresidual, 512 threads and 320: bf16 68.0 us,
// 67.8; fp32 105, 129).
template <int D>
cudaError_t bwd_any(const arx_layer_norm_bwd_args& a, bool vec, unsigned* parts, cudaStream_t st) {
  const uint64_t n = a.cols;
  bool done = true;
  cudaError_t e = cudaSuccess;
  if (vec) {
    if (n <= 256)
      e = bwd<D, 32, 8, 1, 8>(a, parts, &done, st);
    else if (n <= 512)
      e = bwd<D, 32, 8, 2, 8>(a, parts, &done, st);
    else if (n <= 1024)
      e = bwd<D, 64, 4, 2, 8>(a, parts, &done, st);
    else if (n <= 2048)
      e = bwd<D, 128, 2, 2, 8>(a, parts, &done, st);
    else if (n <= 4096)
      e = bwd<D, 256, 1, 2, 8>(a, parts, &done, st);
    else if (n <= 8192)
      e = bwd<D, 512, 1, 2, 8>(a, parts, &done, st);
    else if (n <= 16384)
      e = bwd<D, 512, 1, 4, 8>(a, parts, &done, st);
    else
      done = false;
  } else {
    if (n <= 256)
      e = bwd<D, 32, 8, 8, 1>(a, parts, &done, st);
    else if (n <= 512)
      e = bwd<D, 32, 8, 16, 1>(a, parts, &done, st);
    else if (n <= 1024)
      e = bwd<D, 64, 4, 16, 1>(a, parts, &done, st);
    else if (n <= 2048)
      e = bwd<D, 128, 2, 16, 1>(a, parts, &done, st);
    else if (n <= 4096)
      e = bwd<D, 256, 1, 16, 1>(a, parts, &done, st);
    else if (n <= 5120)
      e = bwd<D, 320, 1, 16, 1>(a, parts, &done, st);
    else if (n <= 8192)
      e = bwd<D, 512, 1, 16, 1>(a, parts, &done, st);
    else if (n <= 16384)
      e = bwd<D, 1024, 1, 16, 1>(a, parts, &done, st);
    else
      done = false;
  }
  if (e != cudaSuccess || done) return e;
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

// An upper bound: kBwdBlocks to an SM, or the chunks of the long form.
size_t norm_bwd_parts(uint64_t rows, uint64_t cols) {
  (void)cols;
  return size_t(rows < 2 * kSms ? rows : 2 * kSms);
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
