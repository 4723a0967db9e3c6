// The end of a sublayer in one kernel: rank-order sum of W bf16 partials,
// bias, dropout, residual, layer norm.
//
// Bound by HBM: (W + 1) row reads and two row writes; run one after the other
// the three operators would write and read the sum and h once more each.  Rows
// off 16 bytes are bound by issue slots: one 2-byte load for each element of
// each slot, and with dropout a generator evaluation for each element where a
// whole unit shares one (W = 4 [1001, 5003]: 35.9 us, with dropout 42.4, the bytes'
// time 10.3).  Rows beyond the registers (8192 columns off 16 bytes, 16384 of whole
// units) do that in each of three passes (W = 4 [300, 20000]: 55.6 and 89.8, bytes 12.4).
#include <cuda_runtime.h>

#include "arx_internal.h"
#include "norm.cuh"
#include "ops_launch.h"

namespace arx {
namespace {

struct ReduceNormArgs {
  const uint16_t* slot[kMaxW];
  const uint16_t *bias, *residual, *weight, *norm_bias;
  uint16_t *h, *y;
  float *mean, *rstd;
  const uint64_t* rng;
  size_t rows, cols;
  float eps, scale, inv_cols;
  uint32_t threshold;
};

// Dropout of the unit's V columns starting at c.
template <int V>
__device__ __forceinline__ void dropout_unit(float (&f)[V], const DropoutState& d, uint32_t c, uint32_t row) {
  if constexpr (V == 8)
    dropout8(f, d, c >> 3, row);
  else
    f[0] = dropout1(f[0], d, c, row);
}

template <int W, int TPR, int RPC, int NV, int V>
__global__ void __launch_bounds__(TPR* RPC) reduce_norm_kernel(const ReduceNormArgs a) {
  __shared__ float buf[RPC][2 * (TPR / 32)];
  dependent_launch_prologue();
  const size_t row = size_t(blockIdx.x) * RPC + threadIdx.x / TPR;
  if (RPC > 1 && row >= a.rows) return;
  const uint32_t cols = uint32_t(a.cols);
  const size_t base = row * a.cols;
  DropoutState d{};
  if (a.threshold) d = load_dropout(a.rng, a.threshold, a.scale);
  float f[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const uint32_t c = row_col<TPR, V>(i);
#pragma unroll
    for (int k = 0; k < V; ++k) f[i][k] = 0.0f;
    if (c >= cols) continue;
    Pack<ARX_BF16, V> p[W], r;
#pragma unroll
    for (int w = 0; w < W; ++w) p[w].load(a.slot[w] + base + c);
    if (a.residual) r.load(a.residual + base + c);
    float v[V];
#pragma unroll
    for (int w = 0; w < W; ++w) {
      p[w].get(v);
#pragma unroll
      for (int k = 0; k < V; ++k) f[i][k] = __fadd_rn(f[i][k], v[k]);
    }
    if (a.bias) {
      load_params<V>(a.bias, ARX_BF16, c, v);
#pragma unroll
      for (int k = 0; k < V; ++k) f[i][k] += v[k];
    }
    if (a.threshold) dropout_unit<V>(f[i], d, c, uint32_t(row));
    if (a.residual) {
      r.get(v);
#pragma unroll
      for (int k = 0; k < V; ++k) f[i][k] += v[k];
    }
    if (a.h) {
      Pack<ARX_BF16, V> o;
      o.set(f[i]);
      o.store(a.h + base + c);
    }
  }
  norm_row<ARX_BF16, TPR, NV, V>(f, cols, a.inv_cols, a.eps, a.weight, a.norm_bias, ARX_BF16, a.y + base,
                                 a.mean ? a.mean + row : nullptr, a.rstd ? a.rstd + row : nullptr,
                                 buf[threadIdx.x / TPR]);
}

// h of one element, before its rounding.
template <int W>
__device__ __forceinline__ float sublayer_sum(const ReduceNormArgs& a, const DropoutState& d, size_t row, size_t c) {
  const size_t e = row * a.cols + c;
  float s = 0.0f;
#pragma unroll
  for (int w = 0; w < W; ++w) s = __fadd_rn(s, widen16(a.slot[w][e]));
  if (a.bias) s += widen16(a.bias[c]);
  if (a.threshold) s = dropout1(s, d, uint32_t(c), uint32_t(row));
  if (a.residual) s += widen16(a.residual[e]);
  return s;
}

// Any row length: one block per row, h computed anew in each of three passes
// and stored, with y, in the last, after its element's last read.
template <int W>
__global__ void __launch_bounds__(512) reduce_norm_long_kernel(const ReduceNormArgs a) {
  __shared__ float buf[2][16];
  dependent_launch_prologue();
  const size_t row = blockIdx.x;
  DropoutState d{};
  if (a.threshold) d = load_dropout(a.rng, a.threshold, a.scale);
  float s = 0.0f;
  for (size_t c = threadIdx.x; c < a.cols; c += 512) s += sublayer_sum<W>(a, d, row, c);
  const float mean = row_sum<512, 1>(s, buf[0]) / float(a.cols);
  float q = 0.0f;
  for (size_t c = threadIdx.x; c < a.cols; c += 512) {
    const float v = sublayer_sum<W>(a, d, row, c) - mean;
    q += v * v;
  }
  const float rstd = 1.0f / sqrtf(row_sum<512, 1>(q, buf[1]) / float(a.cols) + a.eps);
  for (size_t c = threadIdx.x; c < a.cols; c += 512) {
    const float h = sublayer_sum<W>(a, d, row, c);
    float o = (h - mean) * rstd;
    if (a.weight) o *= widen16(a.weight[c]);
    if (a.norm_bias) o += widen16(a.norm_bias[c]);
    if (a.h) a.h[row * a.cols + c] = round_bf16(h);
    a.y[row * a.cols + c] = round_bf16(o);
  }
  if (threadIdx.x == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
}

template <int W, int TPR, int RPC, int NV, int V>
cudaError_t run(const ReduceNormArgs& a, cudaStream_t st) {
  return launch_op(reduce_norm_kernel<W, TPR, RPC, NV, V>, dim3(unsigned((a.rows + RPC - 1) / RPC)), TPR * RPC, 0, st,
                   a);
}

template <int W>
cudaError_t run_w(const ReduceNormArgs& a, bool vec, cudaStream_t st) {
  const size_t n = a.cols;
  // 32 columns to a thread, so that a row's sums and bookkeeping cost few
  // instructions, or 8, for the least time of a row.  Measured, time of 32
  // columns by that of 8:
  //  above 4096 columns  1024 threads to a row fill an SM: from 153 rows on .45 to
  //                      .98 (up to 5120 columns), .6 to 1.1 (8192); up to 152
  //                      rows .85 to 1.2
  //  2049 to 4096        W of 1 and 2 from 609 rows on .87 to 1.13, below to 1.25; 3
  //                      and 4 .92 to 1.25; above, from 2.5 million elements on
  //                      .75 to 1.05, below to 1.2
  //  513 to 2048         W of 1 to 6 .95 to 1.9; 7 and 8 from 2.5 million elements
  //                      on .9 to 1.05, below to 1.8 (fewer warps)
  //  257 to 512          up to 1,216 rows .95 to 1.4, above .75 to 1.15
  // 640 threads to rows of up to 5120 columns, against 1024: aligned, up to 152
  // rows, .65 to .9; off 16 bytes, whose elements are read one by one, .7 to .85
  // from 153 rows on, .95 to 1.1 below.
  const bool work = a.rows * n > uint64_t(4 * 152) * 4096;
  if (vec) {
    if (n <= 256) return run<W, 32, 4, 1, 8>(a, st);
    if (n <= 512 && a.rows > 8 * 152) return run<W, 32, 4, 4, 8>(a, st);
    if constexpr (W > 6) {
      if (n <= 1024 && work) return run<W, 32, 4, 4, 8>(a, st);
      if (n <= 2048 && work) return run<W, 64, 1, 4, 8>(a, st);
    }
    if constexpr (W <= 2 || W > 4)
      if (n > 2048 && n <= 4096 && (W <= 2 ? a.rows > 4 * 152 : work)) return run<W, 128, 1, 4, 8>(a, st);
    if (n <= 1024) return run<W, 128, 1, 1, 8>(a, st);
    if (n <= 2048) return run<W, 256, 1, 1, 8>(a, st);
    if (n <= 4096) return run<W, 512, 1, 1, 8>(a, st);
    if (n <= 8192 && a.rows > 152) return run<W, 256, 1, 4, 8>(a, st);
    if (n <= 5120) return run<W, 640, 1, 1, 8>(a, st);
    if (n <= 8192) return run<W, 1024, 1, 1, 8>(a, st);
    if (n <= 16384) return run<W, 512, 1, 4, 8>(a, st);
  } else {
    if (n <= 256) return run<W, 32, 4, 8, 1>(a, st);
    if (n <= 1024) return run<W, 128, 1, 8, 1>(a, st);
    if (n <= 2048) return run<W, 256, 1, 8, 1>(a, st);
    if (n <= 4096) return run<W, 512, 1, 8, 1>(a, st);
    if (n <= 5120) return run<W, 640, 1, 8, 1>(a, st);
    if (n <= 8192) return run<W, 1024, 1, 8, 1>(a, st);
  }
  return launch_op(reduce_norm_long_kernel<W>, dim3(unsigned(a.rows)), 512, 0, st, a);
}

}  // namespace

cudaError_t launch_reduce_layer_norm(const arx_reduce_layer_norm_args& c, bool vec, cudaStream_t st) {
  ReduceNormArgs a{};
  for (int r = 0; r < c.W; ++r) a.slot[r] = static_cast<const uint16_t*>(c.slots[r]);
  a.bias = static_cast<const uint16_t*>(c.bias);
  a.residual = static_cast<const uint16_t*>(c.residual);
  a.weight = static_cast<const uint16_t*>(c.weight);
  a.norm_bias = static_cast<const uint16_t*>(c.norm_bias);
  a.h = static_cast<uint16_t*>(c.h);
  a.y = static_cast<uint16_t*>(c.y);
  a.mean = c.mean;
  a.rstd = c.rstd;
  a.rng = c.rng;
  a.rows = c.rows;
  a.cols = c.cols;
  a.eps = c.eps;
  a.inv_cols = 1.0f / float(c.cols);
  dropout_constants(c.p, &a.threshold, &a.scale);
  switch (c.W) {
    case 1: return run_w<1>(a, vec, st);
    case 2: return run_w<2>(a, vec, st);
    case 3: return run_w<3>(a, vec, st);
    case 4: return run_w<4>(a, vec, st);
    case 5: return run_w<5>(a, vec, st);
    case 6: return run_w<6>(a, vec, st);
    case 7: return run_w<7>(a, vec, st);
    case 8: return run_w<8>(a, vec, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace arx
