// Activations of the matrix product's epilogue and their derivatives, in fp32.
#pragma once

#include <cstdint>

#include "arx.h"

namespace arx {

constexpr float kSqrtHalf = 0.70710678118654752f;       // 1 / sqrt(2)
constexpr float kInvSqrt2Pi = 0.39894228040143268f;     // 1 / sqrt(2 pi)
constexpr float kSqrt2OverPi = 0.79788456080286536f;    // sqrt(2 / pi)
constexpr float kGeluCubic = 0.044715f;

// 1 / (1 + exp(-z)): exp(-z) overflows to infinity for z below -88, and the
// quotient is then 0, its limit.
__device__ __forceinline__ float logistic(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

// z times its logistic; at z = -infinity, where the product would be NaN, 0.
__device__ __forceinline__ float silu(float z) { return z == -INFINITY ? -0.0f : z * logistic(z); }

// The tanh form of gelu, 0.5 z (1 + tanh(u)) with u = sqrt(2/pi) (z + c z^3),
// is z logistic(2 u).
__device__ __forceinline__ float gelu_tanh(float z) {
  const float u = kSqrt2OverPi * (z + kGeluCubic * z * z * z);
  return z == -INFINITY ? -0.0f : z * logistic(2.0f * u);
}

__device__ __forceinline__ float gelu(float z) {
  return z == -INFINITY ? -0.0f : 0.5f * z * (1.0f + erff(z * kSqrtHalf));
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
      for (int i = 0; i < N; ++i) f[i] = gelu(f[i]);
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

// Phi(z) + z phi(z); at infinite z the second term is 0, its limit.
__device__ __forceinline__ float gelu_grad(float z) {
  const float cdf = 0.5f * (1.0f + erff(z * kSqrtHalf));
  const float pdf = kInvSqrt2Pi * __expf(-0.5f * z * z);
  return cdf + (pdf == 0.0f ? 0.0f : z * pdf);
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
template <int N>
__device__ __forceinline__ void multiply_activation_grad(float (&f)[N], const float (&z)[N], int act) {
  switch (act) {
    case ARX_ACT_RELU:
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = z[i] > 0.0f ? f[i] : 0.0f;
      break;
    case ARX_ACT_GELU:
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] *= gelu_grad(z[i]);
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

}  // namespace arx
