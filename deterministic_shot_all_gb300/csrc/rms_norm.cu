// Root-mean-square norm, forward: h = residual + the rank-order sum of W rows
// (one, of any type, or up to eight bf16 partials), y = h rstd weight, and q,
// y in 8 bits with a scale for each row.
//
// Bound by HBM: each row is read once and each output written once.  A row
// stays in its threads' registers between the pass that sums its squares and
// the pass that uses the sum; the largest |y|, which q's scale needs, is found
// with the sum (see row_most).
#include <cuda_runtime.h>

#include "arx_internal.h"
#include "ops_launch.h"
#include "rms_norm.cuh"

namespace arx {
namespace {

template <int D>
struct RmsArgs {
  using S = typename Elem<D>::S;
  const S* slot[kMaxW];
  const S* residual;
  const void* weight;
  S *h, *y;
  uint8_t* q;
  float *scale, *rstd;
  uint64_t rows, cols, ldx, ldresidual, ldh, ldy, ldq;
  float eps, inv_cols;
  int wdtype;
};

// h of the V columns from c on of a row, before its rounding.
template <int D, int W, int V>
__device__ __forceinline__ void load_sum(const RmsArgs<D>& a, size_t row, size_t c, float (&f)[V]) {
  Pack<D, V> p[W], r;
#pragma unroll
  for (int w = 0; w < W; ++w) p[w].load(a.slot[w] + row * a.ldx + c);
  if (a.residual) r.load(a.residual + row * a.ldresidual + c);
#pragma unroll
  for (int k = 0; k < V; ++k) f[k] = 0.0f;
  float v[V];
#pragma unroll
  for (int w = 0; w < W; ++w) {
    p[w].get(v);
#pragma unroll
    for (int k = 0; k < V; ++k) f[k] = __fadd_rn(f[k], v[k]);
  }
  if (a.residual) {
    r.get(v);
#pragma unroll
    for (int k = 0; k < V; ++k) f[k] += v[k];
  }
}

template <int D, int W, int TPR, int RPC, int NV, int V>
__global__ void __launch_bounds__(TPR* RPC) rms_kernel(const __grid_constant__ RmsArgs<D> a) {
  constexpr int kWarps = TPR / 32;
  __shared__ float buf[RPC][4 * kWarps];
  dependent_launch_prologue();
  const size_t row = size_t(blockIdx.x) * RPC + threadIdx.x / TPR;
  if (RPC > 1 && row >= a.rows) return;  // whole warps; RPC > 1 has one warp per row and no barrier
  const uint32_t cols = uint32_t(a.cols);
  float f[NV][V], g[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const uint32_t c = row_col<TPR, V>(i);
#pragma unroll
    for (int k = 0; k < V; ++k) f[i][k] = 0.0f;
    if (c < cols) load_sum<D, W, V>(a, row, c, f[i]);
  }
  hold_params<TPR, NV, V>(g, a.weight, a.wdtype, cols, 1.0f);
  float s = 0.0f;
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int k = 0; k < V; ++k) s += f[i][k] * f[i][k];  // columns past the end hold 0
    if (a.q)
#pragma unroll
      for (int k = 0; k < V; ++k) m = max(m, magnitude(f[i][k] * g[i][k]));
  }
  if (a.h) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t c = row_col<TPR, V>(i);
      Pack<D, V> o;
      o.set(f[i]);
      if (c < cols) o.store(a.h + row * a.ldh + c);
    }
  }
  float* b = buf[threadIdx.x / TPR];
  row_sum_max<TPR, 1>(s, m, b);
  const float rstd = 1.0f / sqrtf(s * a.inv_cols + a.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < V; ++k) f[i][k] = f[i][k] * rstd * g[i][k];
  float scale = 0.0f;
  if (a.q) {
    bool again;
    float most = row_most(m, rstd, again);
    if (again) {
      m = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (row_col<TPR, V>(i) < cols)
#pragma unroll
          for (int k = 0; k < V; ++k) m = max(m, magnitude(f[i][k]));
      row_sum_max<TPR, 1>(s, m, b + 2 * kWarps);
      most = __uint_as_float(m);
    }
    float inverse;
    scale = row_scale(most, inverse);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t c = row_col<TPR, V>(i);
      float o[V];
#pragma unroll
      for (int k = 0; k < V; ++k) o[k] = f[i][k] * inverse;
      if (c < cols) store_e4m3<V>(a.q + row * a.ldq + c, o);
    }
  }
  if (a.y) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t c = row_col<TPR, V>(i);
      Pack<D, V> o;
      o.set(f[i]);
      if (c < cols) o.store(a.y + row * a.ldy + c);
    }
  }
  if (threadIdx.x % TPR == 0) {
    if (a.q) a.scale[row] = scale;
    if (a.rstd) a.rstd[row] = rstd;
  }
}

// Any row length: one block per row, h computed anew in each pass and stored,
// with y and q, in the last, after its element's last read.
template <int D, int W>
__global__ void __launch_bounds__(512) rms_long_kernel(const __grid_constant__ RmsArgs<D> a) {
  __shared__ float buf[2][32];
  dependent_launch_prologue();
  const size_t row = blockIdx.x;
  float s = 0.0f;
  uint32_t m = 0;
  for (size_t c = threadIdx.x; c < a.cols; c += 512) {
    float h[1];
    load_sum<D, W, 1>(a, row, c, h);
    s += h[0] * h[0];
    if (a.q) m = max(m, magnitude(a.weight ? h[0] * load_param(a.weight, a.wdtype, c) : h[0]));
  }
  row_sum_max<512, 1>(s, m, buf[0]);
  const float rstd = 1.0f / sqrtf(s / float(a.cols) + a.eps);
  float inverse = 0.0f;
  if (a.q) {
    bool again;
    float most = row_most(m, rstd, again);
    if (again) {
      m = 0;
      for (size_t c = threadIdx.x; c < a.cols; c += 512) {
        float h[1];
        load_sum<D, W, 1>(a, row, c, h);
        m = max(m, magnitude(a.weight ? h[0] * rstd * load_param(a.weight, a.wdtype, c) : h[0] * rstd));
      }
      row_sum_max<512, 1>(s, m, buf[1]);
      most = __uint_as_float(m);
    }
    const float scale = row_scale(most, inverse);
    if (threadIdx.x == 0) a.scale[row] = scale;
  }
  if (threadIdx.x == 0 && a.rstd) a.rstd[row] = rstd;
  for (size_t c = threadIdx.x; c < a.cols; c += 512) {
    float h[1];
    load_sum<D, W, 1>(a, row, c, h);
    float v = h[0] * rstd;
    if (a.weight) v *= load_param(a.weight, a.wdtype, c);
    if (a.h) a.h[row * a.ldh + c] = Elem<D>::round(h[0]);
    if (a.y) a.y[row * a.ldy + c] = Elem<D>::round(v);
    if (a.q) a.q[row * a.ldq + c] = uint8_t(round_e4m3x2(v * inverse, 0.0f));
  }
}

template <int D, int W, int TPR, int RPC, int NV, int V>
cudaError_t run(const RmsArgs<D>& a, cudaStream_t st) {
  return launch_op(rms_kernel<D, W, TPR, RPC, NV, V>, dim3(unsigned((a.rows + RPC - 1) / RPC)), TPR * RPC, 0, st, a);
}

template <int D, int W>
cudaError_t run_w(const RmsArgs<D>& a, bool vec, cudaStream_t st) {
  const uint64_t n = a.cols;
  if (vec) {
    if (n <= 256) return run<D, W, 32, 4, 1, 8>(a, st);
    if (n <= 1024) return run<D, W, 128, 1, 1, 8>(a, st);
    if (n <= 2048) return run<D, W, 256, 1, 1, 8>(a, st);
    if (n <= 4096) return run<D, W, 512, 1, 1, 8>(a, st);
    if (n <= 8192) return run<D, W, 1024, 1, 1, 8>(a, st);
    if (n <= 16384) return run<D, W, 512, 1, 4, 8>(a, st);
  } else {
    if (n <= 256) return run<D, W, 32, 4, 8, 1>(a, st);
    if (n <= 1024) return run<D, W, 128, 1, 8, 1>(a, st);
    if (n <= 2048) return run<D, W, 256, 1, 8, 1>(a, st);
    if (n <= 4096) return run<D, W, 512, 1, 8, 1>(a, st);
    if (n <= 8192) return run<D, W, 1024, 1, 8, 1>(a, st);
  }
  return launch_op(rms_long_kernel<D, W>, dim3(unsigned(a.rows)), 512, 0, st, a);
}

template <int D>
cudaError_t rms_norm(const arx_rms_norm_args& c, bool vec, cudaStream_t st) {
  using S = typename Elem<D>::S;
  RmsArgs<D> a{};
  a.slot[0] = static_cast<const S*>(c.x);
  a.residual = static_cast<const S*>(c.residual);
  a.weight = c.weight, a.wdtype = c.wdtype;
  a.h = static_cast<S*>(c.h), a.y = static_cast<S*>(c.y);
  a.q = static_cast<uint8_t*>(c.q), a.scale = c.scale, a.rstd = c.rstd;
  a.rows = c.rows, a.cols = c.cols;
  a.ldx = c.ldx, a.ldresidual = c.ldresidual, a.ldh = c.ldh, a.ldy = c.ldy, a.ldq = c.ldq;
  a.eps = c.eps, a.inv_cols = 1.0f / float(c.cols);
  return run_w<D, 1>(a, vec, st);
}

}  // namespace

cudaError_t launch_rms_norm(const arx_rms_norm_args& c, bool vec, cudaStream_t st) {
  if (c.dtype == ARX_BF16) return rms_norm<ARX_BF16>(c, vec, st);
  if (c.dtype == ARX_F16) return rms_norm<ARX_F16>(c, vec, st);
  return rms_norm<ARX_F32>(c, vec, st);
}

cudaError_t launch_reduce_rms_norm(const arx_reduce_rms_norm_args& c, bool vec, cudaStream_t st) {
  RmsArgs<ARX_BF16> a{};
  for (int r = 0; r < c.W; ++r) a.slot[r] = static_cast<const uint16_t*>(c.slots[r]);
  a.residual = static_cast<const uint16_t*>(c.residual);
  a.weight = c.weight, a.wdtype = ARX_BF16;
  a.h = static_cast<uint16_t*>(c.h), a.y = static_cast<uint16_t*>(c.y);
  a.q = static_cast<uint8_t*>(c.q), a.scale = c.scale, a.rstd = c.rstd;
  a.rows = c.rows, a.cols = c.cols;
  a.ldx = a.ldresidual = a.ldh = a.ldy = c.cols, a.ldq = c.ldq;
  a.eps = c.eps, a.inv_cols = 1.0f / float(c.cols);
  switch (c.W) {
    case 1: return run_w<ARX_BF16, 1>(a, vec, st);
    case 2: return run_w<ARX_BF16, 2>(a, vec, st);
    case 3: return run_w<ARX_BF16, 3>(a, vec, st);
    case 4: return run_w<ARX_BF16, 4>(a, vec, st);
    case 5: return run_w<ARX_BF16, 5>(a, vec, st);
    case 6: return run_w<ARX_BF16, 6>(a, vec, st);
    case 7: return run_w<ARX_BF16, 7>(a, vec, st);
    case 8: return run_w<ARX_BF16, 8>(a, vec, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace arx
