// A row of the root-mean-square norm held in registers, and its output in 8
// bits: shared by the kernels of rms_norm.cu.
#pragma once

#include "norm.cuh"

namespace arx {

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
// with the sum of squares, by the same barrier: within a rounding of it while
// both are normal numbers.  Else (a row of zeros, of values whose squares leave
// the range, with infinities or NaN) `again` says that it has to be taken anew.
__device__ __forceinline__ float row_most(uint32_t m, float rstd, bool& again) {
  const float p = __uint_as_float(m);
  again = !(p > 1e-30f && p < 1e30f && rstd > 1e-18f && rstd < 1e18f);
  return p * rstd;
}

}  // namespace arx
