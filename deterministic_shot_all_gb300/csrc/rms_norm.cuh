// Root-mean-square norm, forward: h = residual + the rank-order sum of W rows
// (one, of any type, or up to eight bf16 partials), y = h rstd weight, and q,
// y in 8 bits with a scale for each row (rms_norm.cu, reduce_rms_norm.cu).
//
// Bound by HBM: each row is read once and each output written once.  A row
// stays in its threads' registers between the pass that sums its squares and
// the pass that uses the sum; the largest |y|, which q's scale needs, is found
// with the sum (see row_most).  [8192, 4096] bf16 with residual and 32-bit weights
// 42.9 us, 6.3 TB/s; W = 4 [1024, 8192] 19.7 us, 6.0 TB/s; 32 rows of 4096 2.1 us.
#pragma once

#include <cuda_runtime.h>

#include <type_traits>

#include "arx_internal.h"
#include "norm.cuh"
#include "ops_launch.h"
#include "pairs.cuh"

namespace arx {
namespace {

constexpr float kE4m3Most = 448.0f;                       // largest e4m3 number
constexpr float kLeastScale = 1.1754943508222875e-38f;    // 2^-126

// Two fp32 -> two e4m3 in 16 bits (lo in bits 0-7), nearest even, at most 448; NaN stays.
__device__ __forceinline__ uint16_t round_e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}

// V consecutive elements of q; V = 8 is one aligned access.
template <int V>
__device__ __forceinline__ void store_e4m3(uint8_t* p, const float (&f)[V]) {
  if constexpr (V == 8) {
    const uint32_t a = round_e4m3x2(f[0], f[1]), b = round_e4m3x2(f[2], f[3]), c = round_e4m3x2(f[4], f[5]),
                   d = round_e4m3x2(f[6], f[7]);
    st_global(reinterpret_cast<uint2*>(p), make_uint2(a | b << 16, c | d << 16));
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) p[k] = uint8_t(round_e4m3x2(f[k], 0.0f));
  }
}

// The largest magnitude of three, NaN if one is.
__device__ __forceinline__ float most3(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Magnitudes as bits: ordered as the numbers are, NaN above infinity, so that an
// integer maximum lets NaN through.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// The sum of s and the largest m over a row's T threads, by one barrier.
// `buf`: 2 T / 32 words of the row's shared memory, not those of its last call.
template <int T, int RPC>
__device__ __forceinline__ void row_sum_max(float& s, uint32_t& m, float* buf) {
  constexpr int kWarps = T / 32;
  s = warp_sum(s);
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if constexpr (T > 32) {
    if ((threadIdx.x & 31) == 0) {
      buf[(threadIdx.x % T) / 32] = s;
      buf[kWarps + (threadIdx.x % T) / 32] = __uint_as_float(m);
    }
    row_barrier<T, RPC>();
    s = buf[0], m = __float_as_uint(buf[kWarps]);
#pragma unroll
    for (int i = 1; i < kWarps; ++i) {
      s += buf[i];
      const uint32_t o = __float_as_uint(buf[kWarps + i]);
      m = m > o ? m : o;
    }
  }
}

// scale of a row of q, and what its elements are multiplied by, from the largest
// |v| of the row.
__device__ __forceinline__ float row_scale(float most, float& inverse) {
  const float s = most / kE4m3Most, scale = s < kLeastScale ? 1.0f : s;
  inverse = 1.0f / scale;
  return scale;
}

// The largest |v| = |h rstd weight| from the largest |h weight|, which is known
// with the sum of squares, by the same barrier: two products in another order,
// within 4 2^-24 of each other while both are normal numbers.  Else (a row of zeros, of values whose squares leave
// the range, with infinities or NaN) `again` says that it has to be taken anew.
__device__ __forceinline__ float row_most(uint32_t m, float rstd, bool& again) {
  const float p = __uint_as_float(m);
  again = !(p > 1e-30f && p < 1e30f && rstd > 1e-18f && rstd < 1e18f);
  return p * rstd;
}

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
  int wdtype, W;
  bool alike;  // rows lie alike in every matrix, to their address modulo 16 bytes, and the weights are 16 bits on 16 bytes
};

// The terms of h at the V columns from c on of a row, and their sum before its
// rounding.
template <int D, int W, int V>
struct Terms {
  Pack<D, V> p[W], r;
  __device__ __forceinline__ void load(const RmsArgs<D>& a, size_t row, size_t c) {
#pragma unroll
    for (int w = 0; w < W; ++w) p[w].load(a.slot[w] + row * a.ldx + c);
    if (a.residual) r.load(a.residual + row * a.ldresidual + c);
  }
  __device__ __forceinline__ void sum(const RmsArgs<D>& a, float (&f)[V]) const {
    float v[V];
#pragma unroll
    for (int k = 0; k < V; ++k) f[k] = 0.0f;
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
};
template <int D, int W, int V>
__device__ __forceinline__ void load_sum(const RmsArgs<D>& a, size_t row, size_t c, float (&f)[V]) {
  Terms<D, W, V> t;
  t.load(a, row, c);
  t.sum(a, f);
}

// Two elements to an instruction, where registers in pairs cost nothing (32-bit
// rows of 1024 threads spilled with them: 608 rows of 8192, 13.1 us against 9.6).
template <int D, int V>
constexpr bool kPairs = V == 8 && D != ARX_F32;

template <int D, int NV, int V>
__device__ __forceinline__ void scale_row(float (&f)[NV][V], float by) {
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < V; k += kPairs<D, V> ? 2 : 1) {
      if constexpr (kPairs<D, V>)
        halves(pair(f[i][k], f[i][k + 1]) * pair(by), f[i][k], f[i][k + 1]);
      else
        f[i][k] *= by;
    }
}

template <int D, int T, int NV, int V>
__device__ __forceinline__ void store_row(typename Elem<D>::S* p, uint32_t cols, const float (&f)[NV][V]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const uint32_t c = row_col<T, V>(i);
    Pack<D, V> o;
    o.set(f[i]);
    if (c < cols) o.store(p + c);
  }
}

// rstd of a row whose h is in `f` and whose weights are in `g`, and, for q, what is
// known of the largest |v|.  (Columns past the end hold 0 in f.)
struct RowSums {
  float rstd, most;
  bool again;  // `most` is not it
};
// `buf`: 4 T / 32 words of the row's shared memory; store_h() stores f while the
// sums are on their way.
template <int D, int T, int RPC, int NV, int V, typename StoreH>
__device__ __forceinline__ RowSums row_statistics(const RmsArgs<D>& a, const float (&f)[NV][V], const float (&g)[NV][V],
                                                  float* buf, const StoreH& store_h) {
  float s = 0.0f, most = 0.0f;
  if constexpr (kPairs<D, V>) {
    Pair sum = pair(0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < V; k += 2) {
        const Pair v = pair(f[i][k], f[i][k + 1]);
        sum = fma2(v, v, sum);
      }
    float other;
    halves(sum, s, other);
    s += other;
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < V; ++k) s += f[i][k] * f[i][k];
  }
  if (a.q) {
#pragma unroll
    for (int i = 0; i < NV * V; i += 2) {
      const int j = i + 1 < NV * V ? i + 1 : i;
      most = most3(most, f[i / V][i % V] * g[i / V][i % V], f[j / V][j % V] * g[j / V][j % V]);
    }
  }
  uint32_t m = __float_as_uint(most);  // not negative
  if (a.h) store_h();
  row_sum_max<T, RPC>(s, m, buf);
  RowSums r;
  r.rstd = 1.0f / sqrtf(s * a.inv_cols + a.eps);
  r.most = 0.0f, r.again = false;
  if (a.q) r.most = row_most(m, r.rstd, r.again);
  return r;
}

// f = f rstd g.
template <int D, int NV, int V>
__device__ __forceinline__ void normalise_row(float (&f)[NV][V], const float (&g)[NV][V], float rstd) {
  scale_row<D, NV, V>(f, rstd);
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < V; k += kPairs<D, V> ? 2 : 1) {
      if constexpr (kPairs<D, V>)
        halves(pair(f[i][k], f[i][k + 1]) * pair(g[i][k], g[i][k + 1]), f[i][k], f[i][k + 1]);
      else
        f[i][k] *= g[i][k];
    }
}

// The largest |v| of the row, v in `f`; has(i, k): is f[i][k] a column of the row?  (Those
// past its end hold 0 times rstd, which is NaN where rstd is infinite.)
template <int T, int RPC, int NV, int V, typename Has>
__device__ __forceinline__ float largest(const RowSums& r, const float (&f)[NV][V], float* buf, const Has& has) {
  if (!r.again) return r.most;
  uint32_t m = 0;
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (has(i, k)) m = max(m, magnitude(f[i][k]));
  row_sum_max<T, RPC>(s, m, buf + 2 * (T / 32));
  return __uint_as_float(m);
}

// The rest of a row.
template <int D, int T, int RPC, int NV, int V>
__device__ __forceinline__ void finish_row(const RmsArgs<D>& a, size_t row, uint32_t cols, float (&f)[NV][V],
                                           const float (&g)[NV][V], float* buf) {
  const RowSums sums = row_statistics<D, T, RPC, NV, V>(
      a, f, g, buf, [&] { store_row<D, T, NV, V>(a.h + row * a.ldh, cols, f); });
  normalise_row<D, NV, V>(f, g, sums.rstd);
  float scale = 0.0f;
  if (a.q) {
    if (a.y) store_row<D, T, NV, V>(a.y + row * a.ldy, cols, f);
    float inverse;
    scale = row_scale(largest<T, RPC, NV, V>(sums, f, buf, [&](int i, int) { return row_col<T, V>(i) < cols; }), inverse);
    scale_row<D, NV, V>(f, inverse);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t c = row_col<T, V>(i);
      if (c < cols) store_e4m3<V>(a.q + row * a.ldq + c, f[i]);
    }
  } else {
    store_row<D, T, NV, V>(a.y + row * a.ldy, cols, f);
  }
  if (threadIdx.x % T == 0) {
    if (a.q) a.scale[row] = scale;
    if (a.rstd) a.rstd[row] = sums.rstd;
  }
}

// Few rows: one block (or a warp of one) to a row, the fewer columns to a
// thread the sooner it ends.
template <int D, int W, int T, int RPC, int NV, int V>
__global__ void __launch_bounds__(T* RPC) rms_kernel(const __grid_constant__ RmsArgs<D> a) {
  __shared__ float buf[RPC][4 * (T / 32)];
  dependent_launch_prologue();
  const size_t row = size_t(blockIdx.x) * RPC + threadIdx.x / T;
  if (RPC > 1 && row >= a.rows) return;  // whole warps; RPC > 1 has one warp per row and no barrier
  const uint32_t cols = uint32_t(a.cols);
  float f[NV][V], g[NV][V];
  // Units whose loads are in flight together.
  constexpr int kWords = (T > 512 ? 20 : 40) / (W + 1), kGroup = V == 8 ? 1 : kWords < 8 ? kWords : 8;
#pragma unroll
  for (int i0 = 0; i0 < NV; i0 += kGroup) {
    Terms<D, W, V> t[kGroup];
#pragma unroll
    for (int i = i0; i < i0 + kGroup && i < NV; ++i)
      if (row_col<T, V>(i) < cols) t[i - i0].load(a, row, row_col<T, V>(i));
#pragma unroll
    for (int i = i0; i < i0 + kGroup && i < NV; ++i) {
#pragma unroll
      for (int k = 0; k < V; ++k) f[i][k] = 0.0f;
      if (row_col<T, V>(i) < cols) t[i - i0].sum(a, f[i]);
    }
  }
  hold_params<T, NV, V>(g, a.weight, a.wdtype, cols, 1.0f);
  finish_row<D, T, 1, NV, V>(a, row, cols, f, g, buf[threadIdx.x / T]);
}

// Many rows of whole aligned units: persistent, the weights in registers and the
// rows coming in through a ring of kRing rows in shared memory, each thread
// copying what it reads itself.
template <int D, int T, int NV, int kRing>
__global__ void __launch_bounds__(T, 1) rms_ring_kernel(const __grid_constant__ RmsArgs<D> a, uint32_t slot) {
  using S = typename Elem<D>::S;
  constexpr int V = 8;
  __shared__ float buf[2][4 * (T / 32)];
  extern __shared__ __align__(16) uint8_t smem[];  // [kRing][slots, residual][slot]
  dependent_launch_prologue();
  const uint32_t cols = uint32_t(a.cols), W = a.W, arrays = W + (a.residual ? 1 : 0);
  const size_t step = gridDim.x;
  size_t row = blockIdx.x;
  const auto start = [&](size_t r, uint32_t at) {  // one group, empty past the last row
    if (r < a.rows) {
      uint8_t* dst = smem + at * arrays * slot;
      for (uint32_t w = 0; w < W; ++w) copy_matrix_row<D, T, NV, V>(dst + w * slot, a.slot[w], a.ldx, r, a.rows, cols);
      if (a.residual) copy_matrix_row<D, T, NV, V>(dst + W * slot, a.residual, a.ldresidual, r, a.rows, cols);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i + 1 < kRing; ++i) start(row + i * step, i);
  float g[NV][V];
  hold_params<T, NV, V>(g, a.weight, a.wdtype, cols, 1.0f);
  uint32_t at = 0;
  int parity = 0;
  for (; row < a.rows; row += step) {
    cp_async_wait<kRing - 2>();
    const uint8_t* base = smem + at * arrays * slot;
    float f[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t c = row_col<T, V>(i);
#pragma unroll
      for (int k = 0; k < V; ++k) f[i][k] = 0.0f;
      if (c >= cols) continue;
      float v[V];
#pragma unroll 4
      for (uint32_t w = 0; w < W; ++w) {
        read_shared<D, V>(base + w * slot + c * sizeof(S), v);
#pragma unroll
        for (int k = 0; k < V; ++k) f[i][k] = __fadd_rn(f[i][k], v[k]);
      }
      if (a.residual) {
        read_shared<D, V>(base + W * slot + c * sizeof(S), v);
#pragma unroll
        for (int k = 0; k < V; ++k) f[i][k] += v[k];
      }
    }
    // The slot of the row before, which this thread has read.
    start(row + (kRing - 1) * step, at == 0 ? kRing - 1 : at - 1);
    finish_row<D, T, 1, NV, V>(a, row, cols, f, g, buf[parity]);
    parity ^= 1;
    at = at + 1 == kRing ? 0 : at + 1;
  }
  cp_async_wait<0>();
}

// Rows off 16 bytes that lie alike in every matrix (contiguous ones of one shape):
// a thread takes the 8 elements of an aligned unit, whichever columns those are,
// so that all but a row's two end units move 16 bytes at a time.  `off`: elements
// of the row's first unit before the row.  The weights, which begin on 16 bytes,
// are the halves of two units, shifted by `off`.
struct Span {
  int c0, cols;  // first column (negative in the first unit), of how many
  __device__ __forceinline__ bool whole() const { return c0 >= 0 && c0 + 8 <= cols; }
  __device__ __forceinline__ bool has(int k) const { return c0 + k >= 0 && c0 + k < cols; }
  __device__ __forceinline__ bool any() const { return c0 < cols; }  // off < 8: no unit ends before the row
};

template <int D>
__device__ __forceinline__ void load_span(Pack<D, 8>& p, const uint16_t* row, const Span& s) {
  if (s.whole()) {
    p.load(row + s.c0);
  } else {
    p.zero();
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (s.has(k)) p.w[k / 2] |= uint32_t(row[s.c0 + k]) << (k % 2 * 16);
  }
}

template <int D>
__device__ __forceinline__ void store_span(uint16_t* row, const float (&f)[8], const Span& s) {
  Pack<D, 8> p;
  p.set(f);
  if (s.whole()) {
    p.store(row + s.c0);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (s.has(k)) row[s.c0 + k] = uint16_t(p.w[k / 2] >> (k % 2 * 16));
  }
}

// 8 parameters of a 16-bit type from column c0 on, where c0 + off is a multiple of 8:
// taken out of the two aligned units around them; 1 without any.
template <int D>
__device__ __forceinline__ void span_params(const void* p, uint32_t off, const Span& s, float (&g)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) g[k] = 1.0f;
  if (!p || !s.any()) return;
  const uint16_t* w = static_cast<const uint16_t*>(p);
  const int u = s.c0 + int(off);
  if (u >= 8 && u + 8 <= s.cols) {
    const uint4 a = *reinterpret_cast<const uint4*>(w + u - 8), b = *reinterpret_cast<const uint4*>(w + u);
    uint32_t v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    // 8 - off elements on, in words by powers of two and then half a word.
    const uint32_t by = 8 - off;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = by & 8 ? v[i + 4] : v[i];
#pragma unroll
    for (int i = 0; i < 6; ++i) v[i] = by & 4 ? v[i + 2] : v[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) v[i] = by & 2 ? v[i + 1] : v[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) Elem<D>::widen2(__funnelshift_r(v[i], v[i + 1], (by & 1) * 16), g[2 * i], g[2 * i + 1]);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (s.has(k)) g[k] = Elem<D>::widen(w[s.c0 + k]);
  }
}

template <int D, int W, int T, int NV>
__global__ void __launch_bounds__(T) rms_span_kernel(const __grid_constant__ RmsArgs<D> a) {
  __shared__ float buf[4 * (T / 32)];
  dependent_launch_prologue();
  const size_t row = blockIdx.x, at = row * a.cols;
  const uint32_t off = uint32_t(reinterpret_cast<uintptr_t>(a.slot[0] + at) & 15) / 2;
  Span s[NV];
  float f[NV][8], g[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    s[i] = {int((i * T + threadIdx.x) * 8) - int(off), int(a.cols)};
#pragma unroll
    for (int k = 0; k < 8; ++k) f[i][k] = 0.0f;
    if (!s[i].any()) continue;
    Terms<D, W, 8> t;
#pragma unroll
    for (int w = 0; w < W; ++w) load_span<D>(t.p[w], a.slot[w] + at, s[i]);
    if (a.residual) load_span<D>(t.r, a.residual + at, s[i]);
    t.sum(a, f[i]);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) span_params<D>(a.weight, off, s[i], g[i]);
  const RowSums sums = row_statistics<D, T, 1, NV, 8>(a, f, g, buf, [&] {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (s[i].any()) store_span<D>(a.h + at, f[i], s[i]);
  });
  normalise_row<D, NV, 8>(f, g, sums.rstd);
  if (a.y) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (s[i].any()) store_span<D>(a.y + at, f[i], s[i]);
  }
  if (a.q) {
    float inverse;
    const float scale = row_scale(largest<T, 1, NV, 8>(sums, f, buf, [&](int i, int k) { return s[i].has(k); }), inverse);
    scale_row<D, NV, 8>(f, inverse);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (s[i].has(k)) a.q[row * a.ldq + s[i].c0 + k] = uint8_t(round_e4m3x2(f[i][k], 0.0f));
    if (threadIdx.x == 0) a.scale[row] = scale;
  }
  if (threadIdx.x == 0 && a.rstd) a.rstd[row] = sums.rstd;
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

template <int D, int W, int T, int RPC, int NV, int V>
cudaError_t run(const RmsArgs<D>& a, cudaStream_t st) {
  return launch_op(rms_kernel<D, W, T, RPC, NV, V>, dim3(unsigned((a.rows + RPC - 1) / RPC)), T * RPC, 0, st, a);
}

// Shared memory that a block's ring may fill; one block fits an SM.
constexpr size_t kBlockRingBytes = 220 * 1024;
constexpr unsigned kSms = 152;

// Four rows in the ring, two where four are too large; *done is false where two
// are as well.
template <int D, int T, int NV>
cudaError_t run_ring(const RmsArgs<D>& a, bool* done, cudaStream_t st) {
  const size_t row = size_t(row_slot(a.cols, sizeof(typename Elem<D>::S), 8)) * (a.W + (a.residual ? 1 : 0));
  const auto with = [&](auto rows) {
    constexpr int kRing = decltype(rows)::value;
    constexpr auto kernel = rms_ring_kernel<D, T, NV, kRing>;
    const cudaError_t e = allow_dynamic_smem<kernel>(kBlockRingBytes);
    if (e != cudaSuccess) return e;
    return launch_op(kernel, dim3(unsigned(a.rows < kSms ? a.rows : kSms)), T, kRing * row, st, a,
                     row_slot(a.cols, sizeof(typename Elem<D>::S), 8));
  };
  *done = true;
  if (4 * row <= kBlockRingBytes) return with(std::integral_constant<int, 4>{});
  if (2 * row <= kBlockRingBytes) return with(std::integral_constant<int, 2>{});
  *done = false;
  return cudaSuccess;
}

// One block to a row or the ring?  Measured, GPU time in microseconds (16-bit rows
// with residual, h and y, 32-bit weights; one row to a block, then the ring):
//   aligned        152 rows       608          2,432        8,192
//   2048 columns   1.6  2.0     2.4  3.0     7.5  9.3    21.9  25.2
//   4096           2.0  2.2     3.5  4.2    14.6 14.7    42.6  42.0
//   5120           2.2  2.4     5.2  5.6    18.2 19.7    55.0  60.1
//   8192           2.7  2.9     8.8  9.5    32.6 29.0     104    90
//   12288          3.5  3.5    16.9 12.9    63.8 37.4     209   118
// The ring by the one row's time: 2500 to 5120 columns, 1,216 rows and more, fp16
// and 32 bits 1.0 to 1.25, bf16 .98 to 1.3; 5121 to 8192, 2,432 rows and more, 16 bits
// .86 to .97 with a residual and .95 to 1.06 without, 32 bits 1.07 to 1.17 and .91 to
// .95; sums of 3 and 4 ranks .86 to 1.0 from 1,216 rows on (4 ranks, 1,024 rows of 8192:
// 22.4 against 19.1), at 4096 columns 1.0; with q, whose largest |y| takes issue slots,
// 1.12 and more, but above 8192 columns .6 to .85 with it and without.  Rows off 16
// bytes, read element by element, took 1.1 to 2 times as long through it.
// The threads to a row: 640 up to 5120 columns (1024: 2,432 rows of 5120, 34.7 us
// against 21.8); above, 512 with two units each (1024: 41.7 against 33.0 at 8192,
// 152 rows alike), but 1024 for 32-bit rows (31.3 against 45.8 us).  A warp to rows
// of up to 512 columns from 1,217 on (10,000 rows: 11.7 against 8.2 us, 608: 1.85
// alike).  Off 16 bytes and above 5120 columns, 512 threads for one and two ranks
// from 305 rows on (8191: 2,432 rows 42 against 56 us, 152: 3.9 against 3.6), else
// 1024 (4 ranks 1.7 times as long with 512); up to 16384 columns 1024 up to 304 rows
// (152 rows of 12001: 5.3 against 10.3 us), above, two passes over the row are as fast.
// By units that lie alike, time by that of elements, above 5120 columns: one rank .7
// to 1.0, two .6 to .9, four to eight .55 to .85 (608 rows of 16001, four ranks: 70.7
// against 37.9 us; 2,432 of 8181: 117 against 68); up to 5120, whose elements fewer
// threads have in flight together, .75 to 2.
template <int D, int W>
cudaError_t run_w(const RmsArgs<D>& a, bool vec, cudaStream_t st) {
  const uint64_t n = a.cols;
  if (vec) {
    bool done = false;
    cudaError_t e = cudaSuccess;
    if (n <= 256) return run<D, W, 32, 4, 1, 8>(a, st);
    if (n <= 512 && a.rows > 8 * kSms) return run<D, W, 32, 4, 2, 8>(a, st);
    if (n <= 1024) return run<D, W, 128, 1, 1, 8>(a, st);
    if (n <= 2048) return run<D, W, 256, 1, 1, 8>(a, st);
    if (n <= 4096) return run<D, W, 512, 1, 1, 8>(a, st);
    if (n <= 5120) return run<D, W, 640, 1, 1, 8>(a, st);
    if (n <= 8192) {
      const bool ring = !a.q && !(D == ARX_F32 && a.residual) && a.rows >= (W > 2 ? 5 : 16) * kSms;
      if (ring && W <= 4) e = run_ring<D, 1024, 1>(a, &done, st);
      if (e != cudaSuccess || done) return e;
      if constexpr (D == ARX_F32) return run<D, W, 1024, 1, 1, 8>(a, st);
      return run<D, W, 512, 1, 2, 8>(a, st);
    }
    if (n <= 16384) {
      if (a.rows > 2 * kSms && W <= 2) e = run_ring<D, 1024, 2>(a, &done, st);
      if (e != cudaSuccess || done) return e;
      if constexpr (W > 2) return run<D, W, 1024, 1, 2, 8>(a, st);
      return run<D, W, 512, 1, 4, 8>(a, st);
    }
  } else {
    if constexpr (D != ARX_F32)
      if (a.alike && n > 5120) {  // (a row may begin 7 elements into its first unit)
        const dim3 grid(unsigned(a.rows));
        if (n + 7 <= 8192) return launch_op(rms_span_kernel<D, W, 512, 2>, grid, 512, 0, st, a);
        if (n + 7 <= 16384) return launch_op(rms_span_kernel<D, W, 1024, 2>, grid, 1024, 0, st, a);
      }
    if (n <= 256) return run<D, W, 32, 4, 8, 1>(a, st);
    if (n <= 512 && a.rows > 8 * kSms) return run<D, W, 64, 1, 8, 1>(a, st);
    if (n <= 1024) return run<D, W, 128, 1, 8, 1>(a, st);
    if (n <= 2048) return run<D, W, 256, 1, 8, 1>(a, st);
    if (n <= 4096) return run<D, W, 512, 1, 8, 1>(a, st);
    if (n <= 5120) return run<D, W, 640, 1, 8, 1>(a, st);
    if constexpr (W <= 2)
      if (n <= 8192 && a.rows > 2 * kSms) return run<D, W, 512, 1, 16, 1>(a, st);
    if (n <= 8192) return run<D, W, 1024, 1, 8, 1>(a, st);
    if (n <= 16384 && a.rows <= 2 * kSms) return run<D, W, 1024, 1, 16, 1>(a, st);
  }
  return launch_op(rms_long_kernel<D, W>, dim3(unsigned(a.rows)), 512, 0, st, a);
}

}  // namespace
}  // namespace arx
