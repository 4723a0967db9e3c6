// Layer norm of rows held in registers: shared by the layer norm kernels and
// by the fused end of the rank-order reduce.
#pragma once

#include "arx_rows.cuh"

namespace arx {

// A row's columns are spread over its TPR threads in units of V: thread t
// holds units t, t + TPR, ..., NV of them, so a warp's accesses are contiguous.
template <int TPR, int V>
__device__ __forceinline__ uint32_t row_col(int i) {
  return (uint32_t(i) * TPR + threadIdx.x % TPR) * V;
}

// Sets mean and rstd of the row and, when `y` is not null, stores its
// normalised elements.  The variance is the mean square about the mean, taken
// in a second pass over the registers: sum(x^2) / n - mean^2 would cancel
// where the mean is large against the spread.
template <int D, int TPR, int NV, int V>
__device__ __forceinline__ void norm_row(const float (&f)[NV][V], uint32_t cols, float eps, const void* weight,
                                         const void* bias, int wdtype, typename Elem<D>::S* y, float* mean_out,
                                         float* rstd_out, float* buf) {
  constexpr int kWarps = TPR / 32;
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < V; ++k) s += f[i][k];  // columns past the end hold 0
  const float mean = row_sum<TPR>(s, buf) / float(cols);
  float q = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (row_col<TPR, V>(i) < cols)
#pragma unroll
      for (int k = 0; k < V; ++k) q += (f[i][k] - mean) * (f[i][k] - mean);
  const float rstd = 1.0f / sqrtf(row_sum<TPR>(q, buf + kWarps) / float(cols) + eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const uint32_t c = row_col<TPR, V>(i);
    if (c >= cols) continue;
    float o[V], p[V];
#pragma unroll
    for (int k = 0; k < V; ++k) o[k] = (f[i][k] - mean) * rstd;
    if (weight) {
      load_params<V>(weight, wdtype, c, p);
#pragma unroll
      for (int k = 0; k < V; ++k) o[k] *= p[k];
    }
    if (bias) {
      load_params<V>(bias, wdtype, c, p);
#pragma unroll
      for (int k = 0; k < V; ++k) o[k] += p[k];
    }
    Pack<D, V> out;
    out.set(o);
    out.store(y + c);
  }
  if (threadIdx.x % TPR == 0) {
    if (mean_out) *mean_out = mean;
    if (rstd_out) *rstd_out = rstd;
  }
}

}  // namespace arx
