// Activations of the matrix product's epilogue and their derivatives, in fp32.
#pragma once

#include <cfloat>
#include <cstdint>

#include "arx.h"
#include "pairs.cuh"

namespace arx {

constexpr float kInvSqrt2Pi = 0.39894228040143268f;     // 1 / sqrt(2 pi)
constexpr float kSqrt2OverPi = 0.79788456080286536f;    // sqrt(2 / pi)
constexpr float kGeluCubic = 0.044715f;
constexpr float kLog2E = 1.4426950408889634f;

// The hardware's base-2 exponential and reciprocal, subnormals to zero: one
// instruction each.  (The forms that keep subnormals take several: silu in the
// epilogue of a [4096, 4096] x [4096, 4096] product took 24 us, now 8.)
__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float reciprocal_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 1 / (1 + 2^y): the power overflows to infinity for y above 128, and the
// quotient is then 0, its limit.
__device__ __forceinline__ float logistic2(float y) { return reciprocal_approx(1.0f + exp2_approx(y)); }
__device__ __forceinline__ float logistic(float z) { return logistic2(-kLog2E * z); }

// z times its logistic; -infinity, whose product with 0 would be NaN, enters it
// as the least finite number.
__device__ __forceinline__ float silu(float z) { return max_nan(z, -FLT_MAX) * logistic(z); }

// The tanh form of gelu, 0.5 z (1 + tanh(u)) with u = sqrt(2/pi) (z + c z^3),
// is z logistic(2 u).
__device__ __forceinline__ float gelu_tanh(float z) {
  constexpr float k = -2.0f * kLog2E * kSqrt2OverPi;
  return max_nan(z, -FLT_MAX) * logistic2(z * fmaf(k * kGeluCubic, z * z, k));
}

// ---- gelu, two elements at a time --------------------------------------------------
//
// Phi and phi from one exponential: Abramowitz and Stegun's 7.1.26, erfc(x) =
// t (a1 + t (a2 + ...)) exp(-x^2) with t = 1 / (1 + p x), within 1.5e-7 of
// erfc for x >= 0; with x = |z| / sqrt(2), tail = Phi(-|z|) = erfc(x) / 2 and
//   gelu(z)  = max(z, 0) - |z| tail,
//   gelu'(z) = 1/2 + sign(z) (1/2 - tail + |z| phi(z)).
// |z| is cut at 30, where tail and phi are 0, so that infinities meet no 0;
// NaN passes.  Products and sums are packed two to an instruction.  (With an
// erf and an exponential of their own the gradient's pass was bound by
// arithmetic: 118 us at [8185, 8192], three times the bytes' time.)
// exp(-a^2 / 2) and Phi(-a) of a = |z| cut at 30.
__device__ __forceinline__ void normal_tail(Pair a, Pair& e, Pair& tail) {
  float x, y;
  halves(a * a * pair(-0.72134752f), x, y);  // log2(e) / 2
  e = pair(exp2_approx(x), exp2_approx(y));
  halves(fma2(a, pair(0.23164190f), pair(1.0f)), x, y);  // 0.3275911 / sqrt(2)
  const Pair t = pair(reciprocal_approx(x), reciprocal_approx(y));
  Pair p = fma2(pair(0.5f * 1.061405429f), t, pair(0.5f * -1.453152027f));
  p = fma2(p, t, pair(0.5f * 1.421413741f));
  p = fma2(p, t, pair(0.5f * -0.284496736f));
  p = fma2(p, t, pair(0.5f * 0.254829592f));
  tail = p * t * e;
}

__device__ __forceinline__ void gelu2(float& z0, float& z1) {
  const Pair a = pair(min_nan(fabsf(z0), 30.0f), min_nan(fabsf(z1), 30.0f));
  Pair e, tail;
  normal_tail(a, e, tail);
  halves(fma2(a * pair(-1.0f), tail, pair(max_nan(z0, 0.0f), max_nan(z1, 0.0f))), z0, z1);
}

// f *= gelu'(z)
__device__ __forceinline__ void gelu_grad2(float& f0, float& f1, float z0, float z1) {
  const Pair a = pair(min_nan(fabsf(z0), 30.0f), min_nan(fabsf(z1), 30.0f));
  Pair e, tail;
  normal_tail(a, e, tail);
  float h0, h1;
  halves(fma2(tail, pair(-1.0f), fma2(a * pair(kInvSqrt2Pi), e, pair(0.5f))), h0, h1);
  f0 *= 0.5f + copysignf(h0, z0);
  f1 *= 0.5f + copysignf(h1, z1);
}

// f[i] = act(f[i]).  The switch is outside the elements' loop: every thread of
// a launch takes the same case.
template <int N>
__device__ __forceinline__ void activate(float (&f)[N], int act) {
  switch (act) {
    case ARX_ACT_RELU:
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = f[i] < 0.0f ? 0.0f : f[i];  // NaN passes
      break;
    case ARX_ACT_GELU:
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        float none = 0.0f;
        gelu2(f[i], i + 1 < N ? f[i + 1 < N ? i + 1 : i] : none);
      }
      break;
    case ARX_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = gelu_tanh(f[i]);
      break;
    case ARX_ACT_SILU:
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = silu(f[i]);
      break;
    default:
      break;
  }
}

// With s = logistic(2 u): s + z s (1 - s) 2 u'; where s (1 - s) is 0 so is
// the term.
__device__ __forceinline__ float gelu_tanh_grad(float z) {
  const float s = logistic(2.0f * kSqrt2OverPi * (z + kGeluCubic * z * z * z));
  const float w = s * (1.0f - s);
  return s + (w == 0.0f ? 0.0f : z * w * (2.0f * kSqrt2OverPi) * (1.0f + 3.0f * kGeluCubic * z * z));
}

__device__ __forceinline__ float silu_grad(float z) {
  const float s = logistic(z);
  const float w = s * (1.0f - s);
  return s + (w == 0.0f ? 0.0f : z * w);
}

// f[i] *= act'(z[i]).
template <int N>  // even
__device__ __forceinline__ void multiply_activation_grad(float (&f)[N], const float (&z)[N], int act) {
  switch (act) {
    case ARX_ACT_RELU:
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = z[i] > 0.0f ? f[i] : 0.0f;
      break;
    case ARX_ACT_GELU:
#pragma unroll
      for (int i = 0; i < N; i += 2) gelu_grad2(f[i], f[i + 1], z[i], z[i + 1]);
      break;
    case ARX_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] *= gelu_tanh_grad(z[i]);
      break;
    case ARX_ACT_SILU:
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] *= silu_grad(z[i]);
      break;
    default:
      break;
  }
}

// f[i] *= act'(z[i]), h[i] *= act(z[i]), with what the two have in common worked out
// once.
template <int N>  // even
__device__ __forceinline__ void multiply_activation_both(float (&f)[N], float (&h)[N], const float (&z)[N], int act) {
  switch (act) {
    case ARX_ACT_RELU:
#pragma unroll
      for (int i = 0; i < N; ++i) {
        f[i] = z[i] > 0.0f ? f[i] : 0.0f;
        h[i] *= z[i] < 0.0f ? 0.0f : z[i];
      }
      break;
    case ARX_ACT_GELU:
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const Pair a = pair(min_nan(fabsf(z[i]), 30.0f), min_nan(fabsf(z[i + 1]), 30.0f));
        Pair e, tail;
        normal_tail(a, e, tail);
        float s0, s1, v0, v1;
        halves(fma2(tail, pair(-1.0f), fma2(a * pair(kInvSqrt2Pi), e, pair(0.5f))), s0, s1);
        halves(fma2(a * pair(-1.0f), tail, pair(max_nan(z[i], 0.0f), max_nan(z[i + 1], 0.0f))), v0, v1);
        f[i] *= 0.5f + copysignf(s0, z[i]);
        f[i + 1] *= 0.5f + copysignf(s1, z[i + 1]);
        h[i] *= v0, h[i + 1] *= v1;
      }
      break;
    case ARX_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < N; ++i) {
        constexpr float k = -2.0f * kLog2E * kSqrt2OverPi;
        const float s = logistic2(z[i] * fmaf(k * kGeluCubic, z[i] * z[i], k)), w = s * (1.0f - s);
        f[i] *= s + (w == 0.0f ? 0.0f : z[i] * w * (2.0f * kSqrt2OverPi) * (1.0f + 3.0f * kGeluCubic * z[i] * z[i]));
        h[i] *= max_nan(z[i], -FLT_MAX) * s;
      }
      break;
    case ARX_ACT_SILU:
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float s = logistic(z[i]), w = s * (1.0f - s);
        f[i] *= s + (w == 0.0f ? 0.0f : z[i] * w);
        h[i] *= max_nan(z[i], -FLT_MAX) * s;
      }
      break;
    default:
#pragma unroll
      for (int i = 0; i < N; ++i) h[i] *= z[i];
      break;
  }
}

}  // namespace arx
