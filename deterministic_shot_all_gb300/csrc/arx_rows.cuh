// Device helpers of the row operators (layer norm, dropout, their joins):
// element types, 8-element vectors, sums over a row's threads, the
// counter-based generator.
//
// Every operator widens its elements to fp32, computes and sums in fp32, and
// rounds once where a result is stored.
#pragma once

#include <cuda_fp16.h>

#include <cstddef>
#include <cstdint>

#include "arx.h"
#include "arx_device.cuh"

namespace arx {

// ---- element types --------------------------------------------------------------

template <int D>
struct Elem;

template <>
struct Elem<ARX_BF16> {
  using S = uint16_t;
  static __device__ __forceinline__ float widen(S v) { return widen16(v); }
  static __device__ __forceinline__ S round(float v) { return round_bf16(v); }
  static __device__ __forceinline__ void widen2(uint32_t w, float& a, float& b) {
    a = widen_lo(w);
    b = widen_hi(w);
  }
  static __device__ __forceinline__ uint32_t round2(float a, float b) { return pack_bf16x2(a, b); }
};

template <>
struct Elem<ARX_F16> {
  using S = uint16_t;
  static __device__ __forceinline__ float widen(S v) { return __half2float(__ushort_as_half(v)); }
  static __device__ __forceinline__ S round(float v) { return __half_as_ushort(__float2half_rn(v)); }
  static __device__ __forceinline__ void widen2(uint32_t w, float& a, float& b) {
    a = widen(uint16_t(w & 0xFFFFu));
    b = widen(uint16_t(w >> 16));
  }
  static __device__ __forceinline__ uint32_t round2(float a, float b) {
    return uint32_t(round(a)) | (uint32_t(round(b)) << 16);
  }
};

template <>
struct Elem<ARX_F32> {
  using S = float;
  static __device__ __forceinline__ float widen(S v) { return v; }
  static __device__ __forceinline__ S round(float v) { return v; }
};

// ---- V consecutive elements of a row ------------------------------------------------
//
// V = 8: one aligned vector access (16 bytes of a 16-bit type, 32 of fp32).
// V = 1: one element, any alignment.  Loads are coherent: every operator may
// write its result over an input it has read.

template <int D, int V>
struct Pack;

template <int D>
struct Pack<D, 8> {
  uint32_t w[4];
  __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0; }
  __device__ __forceinline__ void load(const uint16_t* p) {
    const uint4 v = ld_stream(reinterpret_cast<const uint4*>(p));
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) Elem<D>::widen2(w[i], f[2 * i], f[2 * i + 1]);
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = Elem<D>::round2(f[2 * i], f[2 * i + 1]);
  }
  __device__ __forceinline__ void store(uint16_t* p) const {
    st_global(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
  }
};

template <>
struct Pack<ARX_F32, 8> {
  float w[8];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 0.0f;
  }
  // One 32-byte access per thread: two 16-byte ones would each move half of
  // every 32-byte sector the warp touches.
  __device__ __forceinline__ void load(const float* p) {
    asm volatile("ld.global.L1::no_allocate.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(w[0]), "=f"(w[1]), "=f"(w[2]), "=f"(w[3]), "=f"(w[4]), "=f"(w[5]), "=f"(w[6]),
                   "=f"(w[7])
                 : "l"(p) : "memory");
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = w[i];
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = f[i];
  }
  __device__ __forceinline__ void store(float* p) const {
    asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 :: "l"(p), "f"(w[0]), "f"(w[1]), "f"(w[2]), "f"(w[3]), "f"(w[4]), "f"(w[5]), "f"(w[6]),
                    "f"(w[7])
                 : "memory");
  }
};

template <int D>
struct Pack<D, 1> {
  using S = typename Elem<D>::S;
  S w;
  __device__ __forceinline__ void zero() { w = S(0); }
  __device__ __forceinline__ void load(const S* p) { w = *p; }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = Elem<D>::widen(w); }
  __device__ __forceinline__ void set(const float (&f)[1]) { w = Elem<D>::round(f[0]); }
  __device__ __forceinline__ void store(S* p) const { *p = w; }
};

// ---- parameters (weights, biases and their gradients): the operator's type or fp32 ----
//
// Read by every row and so served from cache; the type is a run-time value
// (a branch that every thread takes alike), not one more template argument.

__device__ __forceinline__ float load_param(const void* p, int dtype, size_t i) {
  if (dtype == ARX_F32) return static_cast<const float*>(p)[i];
  const uint16_t v = static_cast<const uint16_t*>(p)[i];
  return dtype == ARX_BF16 ? Elem<ARX_BF16>::widen(v) : Elem<ARX_F16>::widen(v);
}

__device__ __forceinline__ void store_param(void* p, int dtype, size_t i, float v) {
  if (dtype == ARX_F32)
    static_cast<float*>(p)[i] = v;
  else
    static_cast<uint16_t*>(p)[i] = dtype == ARX_BF16 ? Elem<ARX_BF16>::round(v) : Elem<ARX_F16>::round(v);
}

// V consecutive parameters; V = 8 needs them 16-byte aligned.
template <int V>
__device__ __forceinline__ void load_params(const void* p, int dtype, size_t i, float (&f)[V]) {
  if constexpr (V == 8) {
    if (dtype == ARX_F32) {
      const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
      const float4 a = q[0], b = q[1];
      f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    } else {
      const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (dtype == ARX_BF16)
          Elem<ARX_BF16>::widen2(w[k], f[2 * k], f[2 * k + 1]);
        else
          Elem<ARX_F16>::widen2(w[k], f[2 * k], f[2 * k + 1]);
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) f[k] = load_param(p, dtype, i + k);
  }
}

// ---- sums over the threads of a row ---------------------------------------------
//
// A butterfly within the warp, then the warps' sums in warp order: the same
// order on every run, and every thread gets the same bits.

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}

// Barrier of a row's T threads; RPC rows to a block (a hardware barrier of
// its own for each where there are several).
template <int T, int RPC>
__device__ __forceinline__ void row_barrier() {
  if constexpr (T == 32)
    __syncwarp();
  else if constexpr (RPC == 1)
    __syncthreads();
  else
    asm volatile("bar.sync %0, %1;" :: "r"(1 + threadIdx.x / T), "n"(T) : "memory");
}

// Sums of N values over the T threads of a row, by one barrier.  `buf`:
// N * T / 32 floats of shared memory of the row, not those of the row's last
// call.
template <int T, int RPC, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* buf) {
  constexpr int kWarps = T / 32;
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = warp_sum(v[n]);
  if constexpr (T > 32) {
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int n = 0; n < N; ++n) buf[n * kWarps + (threadIdx.x % T) / 32] = v[n];
    row_barrier<T, RPC>();
#pragma unroll
    for (int n = 0; n < N; ++n) {
      v[n] = buf[n * kWarps];
#pragma unroll
      for (int i = 1; i < kWarps; ++i) v[n] += buf[n * kWarps + i];
    }
  }
}

template <int T, int RPC>
__device__ __forceinline__ float row_sum(float v, float* buf) {
  float a[1] = {v};
  row_sums<T, RPC, 1>(a, buf);
  return a[0];
}

// ---- asynchronous copies by threads -----------------------------------------------

// 16 bytes to shared memory, both addresses aligned: the first `have` from
// global memory, zeros after.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t have) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(have) : "memory");
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// All but the thread's last kGroups groups have landed.
template <int kGroups>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" :: "n"(kGroups) : "memory");
}

// ---- Philox4x32-10 --------------------------------------------------------------
//
// The counter-based generator of Salmon, Moraes, Dror and Shaw, "Parallel
// random numbers: as easy as 1, 2, 3" (SC 2011): ten rounds of two 32 x 32
// multiplies on a 128-bit counter under a 64-bit key.  The counter is
// (column / 8, row, offset low, offset high): its four words are eight 16-bit
// values, one for each column of the group, low halves first, so the value
// of an element depends on its row and column alone -- not on strides, the
// launch or the pass -- and no mask needs to be stored.

__device__ __forceinline__ uint4 philox4x32_10(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3,
                                               uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t p0 = uint64_t(c0) * 0xD2511F53u, p1 = uint64_t(c2) * 0xCD9E8D57u;
    c0 = uint32_t(p1 >> 32) ^ c1 ^ k0;
    c1 = uint32_t(p1);
    c2 = uint32_t(p0 >> 32) ^ c3 ^ k1;
    c3 = uint32_t(p0);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// What dropout with a threshold T = round(65536 p) of at least 1 needs of a
// call: the generator's seed and offset, T and the scale 65536 / (65536 - T).
struct DropoutState {
  uint32_t k0, k1, o0, o1;
  uint32_t below;  // (T << 16) - 1: a value in a word's high half is at least T when the word is above this
  float scale;
};

__device__ __forceinline__ DropoutState load_dropout(const uint64_t* rng, uint32_t threshold, float scale) {
  DropoutState d;
  const uint64_t seed = rng[0], offset = rng[1];
  d.k0 = uint32_t(seed), d.k1 = uint32_t(seed >> 32);
  d.o0 = uint32_t(offset), d.o1 = uint32_t(offset >> 32);
  d.below = uint32_t((uint64_t(threshold) << 16) - 1u), d.scale = scale;  // T = 65536: no word is above
  return d;
}

// The words of the 8 columns of a group.
__device__ __forceinline__ uint4 dropout_random(const DropoutState& d, uint32_t group, uint32_t row) {
  return philox4x32_10(group, row, d.o0, d.o1, d.k0, d.k1);
}

// Whether column 8 * group + k is kept.
__device__ __forceinline__ bool dropout_keeps(const DropoutState& d, const uint4& r, int k) {
  const uint32_t w = k < 4 ? (k < 2 ? r.x : r.y) : (k < 6 ? r.z : r.w);
  return ((k & 1) ? w : w << 16) > d.below;
}

// Dropout of the 8 columns of a group: kept values scaled, the others +0 (a
// selection, so what is dropped may be infinite or NaN).
__device__ __forceinline__ void dropout_apply(float (&f)[8], const DropoutState& d, const uint4& r) {
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] = dropout_keeps(d, r, k) ? f[k] * d.scale : 0.0f;
}

__device__ __forceinline__ void dropout8(float (&f)[8], const DropoutState& d, uint32_t group, uint32_t row) {
  dropout_apply(f, d, dropout_random(d, group, row));
}

// The same for one element.
__device__ __forceinline__ float dropout1(float f, const DropoutState& d, uint32_t col, uint32_t row) {
  const uint4 r = dropout_random(d, col >> 3, row);
  bool keep = false;
#pragma unroll
  for (int k = 0; k < 8; ++k) keep = (int(col & 7u) == k) ? dropout_keeps(d, r, k) : keep;
  return keep ? f * d.scale : 0.0f;
}

}  // namespace arx
