// Matrix products on the tensor cores, with the epilogue of arx_linear.
//
// out[i][j] = act(sum_k P(i, k) Q(j, k) + bias[j]) + residual[i][j], 16-bit
// operands, fp32 accumulation in tensor memory.  The three products of a
// linear layer are this one with other operand layouts: x w^T (both operands
// K-major), dz w (w MN-major) and dz^T x (both MN-major); the copy engine
// brings 64-element boxes into 128-byte-swizzled shared memory either way and
// the descriptors name the layout, so nothing is transposed in memory.
//
// Roles (warps): one copies, one issues the matrix instructions, four read
// the accumulators and run the epilogue; operands pass through a ring of
// stages guarded by mbarriers.  Matrices that the copy engine cannot address
// (rows off 16 bytes) are loaded by 128 more threads into the same swizzled
// stages.
//
// Two forms:
//  wide   persistent blocks over tiles of 128 x 256, two accumulators in tensor
//         memory, so a tile's epilogue runs under the next tile's products;
//  split  for few tiles (decode, small matrices): the output's columns take
//         the 128 accumulator lanes, its few rows the instruction's N, and a
//         cluster of up to 8 blocks splits the contraction; the partials
//         meet in distributed shared memory and are added in block order, the
//         rank-order sum of a one-shot all-reduce.  Bound by reading the
//         weights once.
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>

#include "activation.cuh"
#include "arx_internal.h"
#include "arx_rows.cuh"
#include "ops_launch.h"
#include "tensor_core.cuh"

namespace arx {
namespace {

constexpr uint32_t kLanes = 128;             // rows of P in a tile (accumulator lanes)
constexpr uint32_t kStep = 64;               // contraction elements in a stage
constexpr uint32_t kPBytes = kLanes * 128;   // P's part of a stage
constexpr uint32_t kMaxStages = 12;
constexpr uint32_t kStageBudget = 200 * 1024;  // also keeps one block on an SM: tensor memory is never contended
constexpr uint32_t kLoaders = 128;

struct GemmArgs {
  const uint16_t *p, *q;
  uint64_t ldp, ldq;
  uint32_t P, Q, K;
  uint32_t p_mn, q_mn;
  uint16_t *out, *z;
  const void* bias;
  const uint16_t* residual;
  uint64_t ldout, ldz, ldresidual;
  uint32_t* status;
  int act, wdtype;
  uint32_t bn;         // rows of Q in a tile
  uint32_t stages, stage_bytes;
  uint32_t steps;      // stages' worth of contraction: ceil(K / 64)
  uint32_t split;      // blocks of a cluster that share a tile's contraction
  uint32_t tiles_p, tiles_q;
  uint32_t idesc, tmem_columns;
  uint32_t vec;        // out, z, residual and bias allow 16-byte accesses
};

struct Shared {
  uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], drain;
  uint32_t tmem;
  volatile uint32_t abort;
};

// Position in the ring of stages: slot and the parity its next wait expects.
struct Ring {
  uint32_t slot = 0, phase = 0;
  __device__ __forceinline__ void next(uint32_t stages) {
    if (++slot == stages) slot = 0, phase ^= 1;
  }
};

__device__ __forceinline__ uint32_t addr_of(const void* p) { return shared_address(p); }

// ---- filling a stage -----------------------------------------------------------

__device__ __forceinline__ void copy_operand(uint32_t dst, const CUtensorMap* map, bool mn, uint32_t row0, uint32_t k0,
                                             uint32_t rows, uint32_t bar) {
  if (!mn) {
    tma_load_2d(dst, map, k0, row0, bar);
  } else {
    for (uint32_t r = 0; r < rows; r += 64) tma_load_2d(dst + r * 128, map, row0 + r, k0, bar);
  }
}

// The copy engine's box in plain loads: `rows` rows of 64 elements at
// (row0, col0) of a [nrows, ncols] matrix, zeros outside it, swizzled as the
// copy engine does (16-byte unit u of row r at u ^ (r mod 8)).
__device__ __forceinline__ void load_box(uint8_t* dst, const uint16_t* src, uint64_t ld, uint32_t nrows, uint32_t ncols,
                                         uint32_t row0, uint32_t col0, uint32_t rows, uint32_t tid) {
  for (uint32_t i = tid; i < rows * 8; i += kLoaders) {
    const uint32_t r = i >> 3, u = i & 7u, row = row0 + r, col = col0 + u * 8;
    uint32_t w[4] = {0, 0, 0, 0};
    if (row < nrows) {
      const uint16_t* p = src + row * ld + col;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (col + k < ncols) w[k >> 1] |= uint32_t(p[k]) << (16 * (k & 1));
    }
    *reinterpret_cast<uint4*>(dst + r * 128 + ((u ^ (r & 7u)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

__device__ __forceinline__ void load_operand(uint8_t* dst, const uint16_t* src, uint64_t ld, bool mn, uint32_t nrows,
                                             uint32_t nk, uint32_t row0, uint32_t k0, uint32_t rows, uint32_t tid) {
  if (!mn) {
    load_box(dst, src, ld, nrows, nk, row0, k0, rows, tid);
  } else {
    for (uint32_t r = 0; r < rows; r += 64) load_box(dst + r * 128, src, ld, nk, nrows, k0, row0 + r, 64, tid);
  }
}

// ---- the roles, for one tile -------------------------------------------------------

// One thread (the copy engine) or kLoaders threads.  Returns false after a
// wait ran out.
template <bool kTma>
__device__ __forceinline__ bool fill_tile(const GemmArgs& a, const CUtensorMap* mp, const CUtensorMap* mq, Shared& s,
                                          uint8_t* stages, Ring& ring, uint32_t p0, uint32_t q0, uint32_t first,
                                          uint32_t last, uint32_t tid) {
  for (uint32_t i = first; i < last; ++i) {
    if (!mbar_wait(addr_of(&s.empty[ring.slot]), ring.phase ^ 1, &s.abort)) return false;
    uint8_t* dst = stages + ring.slot * a.stage_bytes;
    const uint32_t bar = addr_of(&s.full[ring.slot]);
    if constexpr (kTma) {
      mbar_arrive_expect(bar, a.stage_bytes);
      copy_operand(addr_of(dst), mp, a.p_mn, p0, i * kStep, kLanes, bar);
      copy_operand(addr_of(dst) + kPBytes, mq, a.q_mn, q0, i * kStep, a.bn, bar);
    } else {
      load_operand(dst, a.p, a.ldp, a.p_mn, a.P, a.K, p0, i * kStep, kLanes, tid);
      load_operand(dst + kPBytes, a.q, a.ldq, a.q_mn, a.Q, a.K, q0, i * kStep, a.bn, tid);
      fence_async_shared();
      mbar_arrive(bar);
    }
    ring.next(a.stages);
  }
  return true;
}

// One thread issues the tile's products into `tmem`.
__device__ __forceinline__ bool multiply_tile(const GemmArgs& a, Shared& s, uint32_t stages, Ring& ring, uint32_t tmem,
                                              uint32_t first, uint32_t last) {
  // A contraction step of 16 is 32 bytes along a K-major row, 16 rows of an
  // MN-major tile; in the descriptors' units of 16 bytes.
  const uint32_t adv_p = a.p_mn ? 128 : 2, adv_q = a.q_mn ? 128 : 2;
  for (uint32_t i = first; i < last; ++i) {
    if (!mbar_wait(addr_of(&s.full[ring.slot]), ring.phase, &s.abort)) return false;
    tmem_fence_after();
    const uint32_t base = stages + ring.slot * a.stage_bytes;
    const uint64_t dp = operand_descriptor(base, kStep * 128), dq = operand_descriptor(base + kPBytes, kStep * 128);
#pragma unroll
    for (uint32_t k = 0; k < kStep / 16; ++k)
      mma_f16(tmem, dp + k * adv_p, dq + k * adv_q, a.idesc, i != first || k != 0);
    mma_commit(addr_of(&s.empty[ring.slot]));
    ring.next(a.stages);
  }
  return true;
}

// Bias, z, activation, residual of 16 consecutive columns of a row.
template <int D>
__device__ __forceinline__ void finish16(const GemmArgs& a, float (&v)[16], uint32_t row, uint32_t col) {
  uint16_t* out = a.out + row * a.ldout + col;
  const uint32_t n = a.Q - col;
  if (a.vec && n >= 16) {
    if (a.bias) {
      float b[8];
#pragma unroll
      for (int h = 0; h < 16; h += 8) {
        load_params<8>(a.bias, a.wdtype, col + h, b);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[h + k] += b[k];
      }
    }
    Pack<D, 8> o;
    if (a.z) {
#pragma unroll
      for (int h = 0; h < 16; h += 8) {
        o.set(reinterpret_cast<const float(&)[8]>(v[h]));
        o.store(a.z + row * a.ldz + col + h);
      }
    }
    activate<16>(v, a.act);
    if (a.residual) {
      float r[8];
#pragma unroll
      for (int h = 0; h < 16; h += 8) {
        o.load(a.residual + row * a.ldresidual + col + h);
        o.get(r);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[h + k] += r[k];
      }
    }
#pragma unroll
    for (int h = 0; h < 16; h += 8) {
      o.set(reinterpret_cast<const float(&)[8]>(v[h]));
      o.store(out + h);
    }
    return;
  }
  if (a.bias)
#pragma unroll
    for (uint32_t k = 0; k < 16; ++k)
      if (k < n) v[k] += load_param(a.bias, a.wdtype, col + k);
  if (a.z)
#pragma unroll
    for (uint32_t k = 0; k < 16; ++k)
      if (k < n) a.z[row * a.ldz + col + k] = Elem<D>::round(v[k]);
  activate<16>(v, a.act);
#pragma unroll
  for (uint32_t k = 0; k < 16; ++k)
    if (k < n) {
      if (a.residual) v[k] += Elem<D>::widen(a.residual[row * a.ldresidual + col + k]);
      out[k] = Elem<D>::round(v[k]);
    }
}

__device__ __forceinline__ void setup(const GemmArgs& a, const CUtensorMap* mp, const CUtensorMap* mq, Shared& s,
                                      bool tma, uint32_t warp) {
  if (threadIdx.x == 0) {
    for (uint32_t i = 0; i < a.stages; ++i) {
      mbar_init(addr_of(&s.full[i]), tma ? 1 : kLoaders);
      mbar_init(addr_of(&s.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(addr_of(&s.acc_full[i]), 1);
      mbar_init(addr_of(&s.acc_empty[i]), 128);
    }
    mbar_init(addr_of(&s.drain), 1);
    s.abort = 0;
    mbar_init_fence();
    if (tma) prefetch_tensor_map(mp), prefetch_tensor_map(mq);
  }
  if (warp == 1) tmem_alloc(addr_of(&s.tmem), a.tmem_columns);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
}

// Every thread, after its role.  When a wait ran out, the copies and the
// matrix instructions still in flight are waited for, again with a bound,
// before the block's memory is given up.  `ring`, `issued`: the copying
// thread's next stage and an upper bound of the stages it filled.
__device__ __forceinline__ void finish_block(const GemmArgs& a, Shared& s, uint32_t warp, uint32_t lane, bool tma,
                                             Ring ring, uint32_t issued) {
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (s.abort) {
    volatile uint32_t own = 0;
    if (tma && threadIdx.x == 0) {
      for (uint32_t i = 0; i < issued && i < a.stages; ++i) {
        if (ring.slot == 0) ring.slot = a.stages, ring.phase ^= 1;
        --ring.slot;
        mbar_wait(addr_of(&s.full[ring.slot]), ring.phase, &own);
      }
    }
    if (warp == 1 && lane == 0) {
      mma_commit(addr_of(&s.drain));
      mbar_wait(addr_of(&s.drain), 0, &own);
    }
    if (threadIdx.x == 0 && a.status) *a.status = uint32_t(ARX_ETIMEOUT) | (12u << 8);
    __syncthreads();
  }
  if (warp == 1) tmem_free(s.tmem, a.tmem_columns);
}

template <bool kTma>
constexpr uint32_t kGemmThreads = kTma ? 192 : 192 + kLoaders;

// Tile order: bands of 8 row tiles, down the band first, so that the blocks
// at work at one time share operands in L2.
__device__ __forceinline__ void tile_at(const GemmArgs& a, uint32_t t, uint32_t& tp, uint32_t& tq) {
  const uint32_t band = 8u * a.tiles_q, b = t / band, in = t - b * band;
  const uint32_t rows = a.tiles_p - 8u * b < 8u ? a.tiles_p - 8u * b : 8u;
  tq = in / rows;
  tp = 8u * b + (in - tq * rows);
}

template <int D, bool kTma>
__global__ void __launch_bounds__(kGemmThreads<kTma>, 1)
    gemm_wide_kernel(const __grid_constant__ GemmArgs a, const __grid_constant__ CUtensorMap mp,
                     const __grid_constant__ CUtensorMap mq) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared s;
  uint8_t* stages = smem_raw + ((1024u - (addr_of(smem_raw) & 1023u)) & 1023u);
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  setup(a, &mp, &mq, s, kTma, warp);
  dependent_launch_prologue();
  const uint32_t tiles = a.tiles_p * a.tiles_q;

  Ring ring;
  uint32_t issued = 0;
  if (kTma ? threadIdx.x == 0 : warp >= 6) {
    for (uint32_t t = blockIdx.x; t < tiles; t += gridDim.x) {
      uint32_t tp, tq;
      tile_at(a, t, tp, tq);
      issued = a.stages;
      if (!fill_tile<kTma>(a, &mp, &mq, s, stages, ring, tp * kLanes, tq * a.bn, 0, a.steps,
                           threadIdx.x - (kTma ? 0 : 192)))
        break;
    }
  } else if (warp == 1 && lane == 0 && a.steps > 0) {
    uint32_t n = 0;
    for (uint32_t t = blockIdx.x; t < tiles; t += gridDim.x, ++n) {
      const uint32_t b = n & 1, use = n >> 1;
      if (!mbar_wait(addr_of(&s.acc_empty[b]), (use & 1) ^ 1, &s.abort)) break;
      tmem_fence_after();
      if (!multiply_tile(a, s, addr_of(stages), ring, s.tmem + b * 256, 0, a.steps)) break;
      mma_commit(addr_of(&s.acc_full[b]));
    }
  } else if (warp >= 2 && warp < 6) {
    const uint32_t quarter = warp & 3;  // the accumulator lanes this warp may read
    uint32_t n = 0;
    for (uint32_t t = blockIdx.x; t < tiles; t += gridDim.x, ++n) {
      uint32_t tp, tq;
      tile_at(a, t, tp, tq);
      const uint32_t b = n & 1, use = n >> 1;
      if (a.steps > 0) {
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(addr_of(&s.acc_full[b]), use & 1, &s.abort))) break;
        tmem_fence_after();
      }
      const uint32_t row = tp * kLanes + quarter * 32 + lane, col0 = tq * a.bn;
      for (uint32_t c = 0; c < a.bn && col0 + c < a.Q; c += 16) {
        float v[16];
        if (a.steps > 0)
          tmem_load16(s.tmem + b * 256 + c + (quarter * 32 << 16), v);
        else
#pragma unroll
          for (int k = 0; k < 16; ++k) v[k] = 0.0f;
        if (row < a.P) finish16<D>(a, v, row, col0 + c);
        __syncwarp();
      }
      tmem_fence_before();
      mbar_arrive(addr_of(&s.acc_empty[b]));
    }
  }
  __syncwarp();
  finish_block(a, s, warp, lane, kTma, ring, issued);
}

// One tile per cluster; block r of the cluster takes the r-th share of the
// contraction.  P's rows are the output's columns here, Q's rows its rows.
template <int D, bool kTma>
__global__ void __launch_bounds__(kGemmThreads<kTma>, 1)
    gemm_split_kernel(const __grid_constant__ GemmArgs a, const __grid_constant__ CUtensorMap mp,
                      const __grid_constant__ CUtensorMap mq) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared s;
  uint8_t* stages = smem_raw + ((1024u - (addr_of(smem_raw) & 1023u)) & 1023u);
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  setup(a, &mp, &mq, s, kTma, warp);
  dependent_launch_prologue();
  const uint32_t rank = blockIdx.x % a.split, tile = blockIdx.x / a.split;
  const uint32_t tp = tile % a.tiles_p, tq = tile / a.tiles_p;
  const uint32_t p0 = tp * kLanes, q0 = tq * a.bn;
  const uint32_t share = (a.steps + a.split - 1) / a.split;
  const uint32_t first = rank * share < a.steps ? rank * share : a.steps;
  const uint32_t last = first + share < a.steps ? first + share : a.steps;
  float* part = reinterpret_cast<float*>(stages);  // [bn][128 lanes], once the stages are done with

  Ring ring;
  if (kTma ? threadIdx.x == 0 : warp >= 6) {
    fill_tile<kTma>(a, &mp, &mq, s, stages, ring, p0, q0, first, last, threadIdx.x - (kTma ? 0 : 192));
  } else if (warp == 1 && lane == 0 && first < last) {
    if (multiply_tile(a, s, addr_of(stages), ring, s.tmem, first, last)) mma_commit(addr_of(&s.acc_full[0]));
  } else if (warp >= 2 && warp < 6) {
    const uint32_t quarter = warp & 3;
    bool ok = true;
    if (first < last) {
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(addr_of(&s.acc_full[0]), 0, &s.abort));
      tmem_fence_after();
    }
    if (ok)
      for (uint32_t c = 0; c < a.bn; c += 16) {
        float v[16];
        if (first < last)
          tmem_load16(s.tmem + c + (quarter * 32 << 16), v);
        else
#pragma unroll
          for (int k = 0; k < 16; ++k) v[k] = 0.0f;
#pragma unroll
        for (int k = 0; k < 16; ++k) part[(c + k) * kLanes + quarter * 32 + lane] = v[k];
      }
  }
  __syncthreads();
  cluster_arrive_release();
  cluster_wait();

  // The tile's elements (column of the output = lane, row = Q's row) are
  // shared out over the cluster's blocks; each is the sum of the partials in
  // block order.
  const uint32_t nq = a.Q - q0 < a.bn ? a.Q - q0 : a.bn;
  const uint32_t total = nq * kLanes;
  const uint32_t per = ((total + a.split - 1) / a.split + 31) & ~31u;
  const uint32_t end = (rank + 1) * per < total ? (rank + 1) * per : total;
  const uint32_t at = addr_of(part);
  for (uint32_t i = rank * per + threadIdx.x; i < end; i += kGemmThreads<kTma>) {
    const uint32_t j = p0 + (i & (kLanes - 1)), row = q0 + i / kLanes;
    float v = 0.0f;
    for (uint32_t r = 0; r < a.split; ++r) v += ld_cluster_f32(cluster_peer_address(at + i * 4, r));
    if (j >= a.P) continue;
    if (a.bias) v += load_param(a.bias, a.wdtype, j);
    if (a.z) a.z[row * a.ldz + j] = Elem<D>::round(v);
    float f[1] = {v};
    activate<1>(f, a.act);
    if (a.residual) f[0] += Elem<D>::widen(a.residual[row * a.ldresidual + j]);
    a.out[row * a.ldout + j] = Elem<D>::round(f[0]);
  }
  __syncwarp();
  cluster_arrive_release();  // no block leaves while a peer reads its partials
  cluster_wait();
  finish_block(a, s, warp, lane, kTma, ring, last - first);
}

// ---- host side ---------------------------------------------------------------------

// cuTensorMapEncodeTiled, looked up once through the runtime (the library
// links no driver library).
PFN_cuTensorMapEncodeTiled_v12000 encode_function(cudaError_t* err) {
  static std::atomic<void*> cached{nullptr};
  void* f = cached.load(std::memory_order_acquire);
  if (!f) {
    cudaDriverEntryPointQueryResult q{};
    *err = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q);
    if (*err != cudaSuccess) return nullptr;
    if (q != cudaDriverEntryPointSuccess || !f) {
      *err = cudaErrorSymbolNotFound;
      return nullptr;
    }
    cached.store(f, std::memory_order_release);
  }
  return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
}

// Map of an operand: boxes of 64 elements along its rows, `box_rows` rows.
cudaError_t encode(CUtensorMap* m, const uint16_t* base, uint64_t ld, uint64_t nrows, uint64_t ncols, uint32_t box_rows,
                   bool bf16) {
  cudaError_t err = cudaSuccess;
  auto f = encode_function(&err);
  if (!f) return err;
  const cuuint64_t dims[2] = {ncols, nrows};
  const cuuint64_t strides[1] = {(nrows > 1 ? ld : (ncols + 7) / 8 * 8) * 2};
  const cuuint32_t box[2] = {64, box_rows}, el[2] = {1, 1};
  const CUresult r = f(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                       const_cast<uint16_t*>(base), dims, strides, box, el, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

bool copyable(const uint16_t* p, uint64_t ld, uint64_t nrows) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (nrows <= 1 || ld % 8 == 0);
}

// Dynamic shared memory above 48 KB is granted per kernel and device.
template <auto kKernel>
cudaError_t allow_smem() {
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kStageBudget + 1024));
  if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev].store(true, std::memory_order_release);
  return e;
}

template <int D, bool kTma>
cudaError_t launch_wide(const GemmArgs& a, const CUtensorMap& mp, const CUtensorMap& mq, int sms, cudaStream_t st) {
  cudaError_t e = allow_smem<gemm_wide_kernel<D, kTma>>();
  if (e != cudaSuccess) return e;
  const uint32_t tiles = a.tiles_p * a.tiles_q;
  return launch_op(gemm_wide_kernel<D, kTma>, dim3(tiles < uint32_t(sms) ? tiles : uint32_t(sms)),
                   kGemmThreads<kTma>, kStageBudget + 1024, st, a, mp, mq);
}

template <int D, bool kTma>
cudaError_t launch_split(const GemmArgs& a, const CUtensorMap& mp, const CUtensorMap& mq, cudaStream_t st) {
  cudaError_t e = allow_smem<gemm_split_kernel<D, kTma>>();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.tiles_p * a.tiles_q * a.split);
  cfg.blockDim = dim3(kGemmThreads<kTma>);
  cfg.dynamicSmemBytes = kStageBudget + 1024;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, gemm_split_kernel<D, kTma>, a, mp, mq);
  return e != cudaSuccess ? e : cudaGetLastError();
}

uint32_t ceil_div(uint64_t a, uint64_t b) { return uint32_t((a + b - 1) / b); }

}  // namespace

cudaError_t launch_gemm(const GemmCall& c, cudaStream_t st) {
  cudaError_t err = cudaSuccess;
  const int sms = current_sm_count(&err);
  if (sms < 1) return err;
  GemmArgs a{};
  a.out = static_cast<uint16_t*>(c.out);
  a.z = static_cast<uint16_t*>(c.z);
  a.bias = c.bias;
  a.residual = static_cast<const uint16_t*>(c.residual);
  a.ldout = c.ldout, a.ldz = c.ldz, a.ldresidual = c.ldresidual;
  a.status = c.status;
  a.act = c.act, a.wdtype = c.wdtype;
  a.K = uint32_t(c.k);
  a.steps = ceil_div(c.k, kStep);

  const auto aligned = [](const void* p, uint64_t ld) {
    return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0);
  };
  a.vec = aligned(a.out, a.ldout) && aligned(a.z, a.ldz) && aligned(a.residual, a.ldresidual) && aligned(a.bias, 8);

  // Wide tiles when they occupy most of the SMs, else the split form.
  const bool wide = uint64_t(ceil_div(c.rows, kLanes)) * ceil_div(c.cols, 256) >= 100;
  const auto *cp = static_cast<const uint16_t*>(c.p), *cq = static_cast<const uint16_t*>(c.q);
  if (wide) {
    a.p = cp, a.q = cq, a.ldp = c.ldp, a.ldq = c.ldq, a.p_mn = c.p_mn, a.q_mn = c.q_mn;
    a.P = uint32_t(c.rows), a.Q = uint32_t(c.cols);
    a.bn = 256;
    a.split = 1;
    a.tmem_columns = 512;
  } else {
    a.p = cq, a.q = cp, a.ldp = c.ldq, a.ldq = c.ldp, a.p_mn = c.q_mn, a.q_mn = c.p_mn;
    a.P = uint32_t(c.cols), a.Q = uint32_t(c.rows);
    a.bn = a.q_mn ? 64 : 16;
    while (a.bn < a.Q && a.bn < 256) a.bn *= 2;
    a.tmem_columns = a.bn < 32 ? 32 : a.bn;
    const uint32_t tiles = ceil_div(a.P, kLanes) * ceil_div(a.Q, a.bn);
    a.split = 1;
    while (a.split < 8 && 2 * a.split * tiles <= uint32_t(sms) && 2 * a.split <= a.steps) a.split *= 2;
  }
  a.tiles_p = ceil_div(a.P, kLanes);
  a.tiles_q = ceil_div(a.Q, a.bn);
  a.stage_bytes = kPBytes + a.bn * 128;
  a.stages = kStageBudget / a.stage_bytes;
  if (a.stages > kMaxStages) a.stages = kMaxStages;
  a.idesc = mma_descriptor(c.dtype == ARX_BF16, a.p_mn, a.q_mn, kLanes, a.bn);

  const uint64_t p_rows = a.p_mn ? a.K : a.P, q_rows = a.q_mn ? a.K : a.Q;
  const bool tma = a.K > 0 && copyable(a.p, a.ldp, p_rows) && copyable(a.q, a.ldq, q_rows);
  CUtensorMap mp{}, mq{};
  const bool bf16 = c.dtype == ARX_BF16;
  if (tma) {
    err = encode(&mp, a.p, a.ldp, p_rows, a.p_mn ? a.P : a.K, a.p_mn ? 64 : kLanes, bf16);
    if (err != cudaSuccess) return err;
    err = encode(&mq, a.q, a.ldq, q_rows, a.q_mn ? a.Q : a.K, a.q_mn ? 64 : a.bn, bf16);
    if (err != cudaSuccess) return err;
  }
  if (wide) {
    if (bf16) return tma ? launch_wide<ARX_BF16, true>(a, mp, mq, sms, st) : launch_wide<ARX_BF16, false>(a, mp, mq, sms, st);
    return tma ? launch_wide<ARX_F16, true>(a, mp, mq, sms, st) : launch_wide<ARX_F16, false>(a, mp, mq, sms, st);
  }
  if (bf16) return tma ? launch_split<ARX_BF16, true>(a, mp, mq, st) : launch_split<ARX_BF16, false>(a, mp, mq, st);
  return tma ? launch_split<ARX_F16, true>(a, mp, mq, st) : launch_split<ARX_F16, false>(a, mp, mq, st);
}

}  // namespace arx
