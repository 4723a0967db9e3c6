// Layer norm of rows held in registers: shared by the layer norm kernels and
// by the fused end of the rank-order reduce.
#pragma once

#include "arx_rows.cuh"
#include "spans.h"

namespace arx {

// A row's columns are spread over its TPR threads in units of V: thread t
// holds units t, t + TPR, ..., NV of them, so a warp's accesses are contiguous.
template <int TPR, int V>
__device__ __forceinline__ uint32_t row_col(int i) {
  return (uint32_t(i) * TPR + threadIdx.x % TPR) * V;
}

// ---- rows through shared memory --------------------------------------------------------
//
// The persistent kernels bring rows in by asynchronous 16-byte copies, some
// rows ahead.  Rows off 16 bytes are copied as the aligned units that cover
// them, clipped to the matrix, and read element by element (V = 1); of rows in
// whole aligned units (V = 8) each thread copies what it reads itself, so that
// a row needs no barrier but those of its sums.

// Copies the aligned units that cover [at, at + bytes) to dst, thread t units
// t, t + T, ...; nothing outside [lo, hi) is read.
template <int T>
__device__ __forceinline__ void copy_row(uint8_t* dst, uintptr_t at, uint32_t bytes, uintptr_t lo, uintptr_t hi) {
  const uintptr_t first = first_unit(at);
  const uint32_t units = row_units(at, bytes);
  for (uint32_t u = threadIdx.x % T; u < units; u += T) {
    const uintptr_t src = first + 16 * u;
    if (src >= lo) {
      cp_async16(shared_address(dst + 16 * u), reinterpret_cast<const void*>(src), unit_bytes(src, hi));
    } else {  // the matrix begins inside the unit
      for (uintptr_t i = lo; i < src + 16 && i < hi; i += 2)
        *reinterpret_cast<uint16_t*>(dst + 16 * u + (i - src)) = *reinterpret_cast<const uint16_t*>(i);
    }
  }
}

// Row `row` of a [rows, cols] matrix to `dst`.
template <int D, int T, int NV, int V>
__device__ __forceinline__ void copy_matrix_row(uint8_t* dst, const typename Elem<D>::S* m, uint64_t ld, size_t row,
                                                size_t rows, uint32_t cols) {
  constexpr uint32_t kSize = sizeof(typename Elem<D>::S);
  if constexpr (V == 8) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t c = row_col<T, V>(i);
      if (c < cols)
#pragma unroll
        for (uint32_t h = 0; h < 8 * kSize; h += 16)
          cp_async16(shared_address(dst + c * kSize + h), reinterpret_cast<const uint8_t*>(m + row * ld + c) + h, 16);
    }
  } else {
    copy_row<T>(dst, reinterpret_cast<uintptr_t>(m + row * ld), cols * kSize, reinterpret_cast<uintptr_t>(m),
                reinterpret_cast<uintptr_t>(m + (rows - 1) * ld + cols));
  }
}

// Where the row's first element lies in its copy.
template <int V>
__device__ __forceinline__ uint32_t row_offset(const void* row) {
  return V == 1 ? uint32_t(reinterpret_cast<uintptr_t>(row) & 15) : 0;
}

// Bytes of a row's copy.
inline uint32_t row_slot(uint64_t cols, size_t size, int V) {
  return uint32_t((cols * size + (V == 1 ? 30 : 0) + 15) / 16 * 16);
}

template <int D, int V>
__device__ __forceinline__ void read_shared(const uint8_t* p, float (&f)[V]) {
  using S = typename Elem<D>::S;
  if constexpr (V == 1) {
    f[0] = Elem<D>::widen(*reinterpret_cast<const S*>(p));
  } else if constexpr (D == ARX_F32) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    Elem<D>::widen2(v.x, f[0], f[1]);
    Elem<D>::widen2(v.y, f[2], f[3]);
    Elem<D>::widen2(v.z, f[4], f[5]);
    Elem<D>::widen2(v.w, f[6], f[7]);
  }
}

// A row's parameters in registers, `missing` where there are none.
template <int T, int NV, int V>
__device__ __forceinline__ void hold_params(float (&g)[NV][V], const void* p, int dtype, uint32_t cols, float missing) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const uint32_t c = row_col<T, V>(i);
#pragma unroll
    for (int k = 0; k < V; ++k) g[i][k] = missing;
    if (p && c < cols) load_params<V>(p, dtype, c, g[i]);
  }
}

// ---- a row held in registers -------------------------------------------------------------

// Sets mean and rstd of the row and, when `y` is not null, stores its
// normalised elements.  The variance is the mean square about the mean, taken
// in a second pass over the registers: sum(x^2) / n - mean^2 would cancel
// where the mean is large against the spread.
template <int D, int TPR, int NV, int V>
__device__ __forceinline__ void norm_row(const float (&f)[NV][V], uint32_t cols, float inv_cols, float eps, const void* weight,
                                         const void* bias, int wdtype, typename Elem<D>::S* y, float* mean_out,
                                         float* rstd_out, float* buf) {
  constexpr int kWarps = TPR / 32;
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < V; ++k) s += f[i][k];  // columns past the end hold 0
  const float mean = row_sum<TPR, 1>(s, buf) * inv_cols;
  float q = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (row_col<TPR, V>(i) < cols)
#pragma unroll
      for (int k = 0; k < V; ++k) q += (f[i][k] - mean) * (f[i][k] - mean);
  const float rstd = 1.0f / sqrtf(row_sum<TPR, 1>(q, buf + kWarps) * inv_cols + eps);
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
