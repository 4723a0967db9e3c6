// Launchers of the operators around the reduce, between their argument checks
// (ops.cu) and their kernels.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstddef>
#include <cstdint>

#include "arx.h"

namespace arx {

// Launch as a programmatic dependent of the stream's previous kernel (every
// kernel waits for it before it touches memory: dependent_launch_prologue).
template <typename... P, typename... A>
cudaError_t launch_op(void (*k)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Dynamic shared memory above 48 KB is granted per kernel and device.
template <auto kKernel>
cudaError_t allow_dynamic_smem(size_t bytes) {
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
  if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev].store(true, std::memory_order_release);
  return e;
}

// `vec`: every row of every matrix, and every vector of parameters, may be
// accessed in aligned units of 8 elements, and the columns are whole units.
cudaError_t launch_layer_norm(const arx_layer_norm_args& a, bool vec, cudaStream_t st);
cudaError_t launch_layer_norm_bwd(const arx_layer_norm_bwd_args& a, bool vec, cudaStream_t st);
// Partial rows that the backward pass writes for each of its two sums.
size_t norm_bwd_parts(uint64_t rows, uint64_t cols);

// threshold and scale of a dropout probability (see arx.h).
void dropout_constants(double p, uint32_t* threshold, float* scale);
cudaError_t launch_dropout_add(const arx_dropout_add_args& a, bool vec, cudaStream_t st);
cudaError_t launch_dropout_add_bwd(const arx_dropout_add_bwd_args& a, bool vec, cudaStream_t st);
cudaError_t launch_reduce_layer_norm(const arx_reduce_layer_norm_args& a, bool vec, cudaStream_t st);

// dz = dout * act'(z) and the column sums of dz (the products' first step).
struct ActGradCall {
  const void *dout, *z;  // z null: dz = dout
  void* dz;              // null: sums only
  void* dbias;           // null: dz only
  float* part;           // column_parts(rows, cols) x cols floats
  uint64_t rows, cols, lddout, ldz, lddz;
  int act, dtype, wdtype;
};
cudaError_t launch_act_grad(const ActGradCall& c, bool vec, cudaStream_t st);
// Partial rows of the column sums of a [rows, cols] matrix.
size_t column_parts(uint64_t rows, uint64_t cols);

// out[c] = sum over i < parts of p[i][c], in order, for one or two (p, out)
// pairs; a null out is skipped, parts == 0 stores zeros.
cudaError_t launch_column_sum(const float* p0, unsigned parts, uint64_t cols, void* out0, const float* p1,
                              void* out1, int dtype, cudaStream_t st);

// One matrix product out = epilogue(P Q^T) on the tensor cores (see linear.cu).
struct GemmCall {
  const void *p, *q;      // operands, 16-bit
  bool p_mn, q_mn;        // false: element (i, k) at p[i * ld + k]; true: at p[k * ld + i]
  uint64_t ldp, ldq;
  uint64_t rows, cols, k; // of the product; k the contraction
  void* out;
  void* z;
  const void* bias;       // [cols]
  const void* residual;
  uint64_t ldout, ldz, ldresidual;
  int act, dtype, wdtype;
  uint32_t* status;
  uint32_t wait_ns;       // limit of a kernel's wait for its own copies and products
  void* copies;           // gemm_copies_bytes(c) bytes, or null
};
cudaError_t launch_gemm(const GemmCall& c, cudaStream_t st);
// Bytes for copies of the operands whose rows are off 16 bytes, 0 where the
// product is faster without.
size_t gemm_copies_bytes(const GemmCall& c);

// Copies of 16-bit matrices: rows of `cols` elements from `ld` to `ld_dst`
// (a multiple of 2, at least cols) apart, dst on 4 bytes.
struct Realign {
  const uint16_t* src;
  uint16_t* dst;
  uint64_t rows, ld, ld_dst;
  int64_t cols;
};
struct RealignPair {
  Realign m[2];
  int n;
};
cudaError_t launch_realign(const RealignPair& pair, cudaStream_t st);

}  // namespace arx
