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
// (rows off 16 bytes) are loaded by 512 more threads into the same swizzled
// stages.
//
// Three forms:
//  vector one to four rows (decode): dot products on the CUDA cores, see
//         dot_kernel; the tensor cores' set-up would cost more than the work.
//  wide   persistent pairs of blocks over tiles of 256 x 256 (one instruction
//         spans both SMs, each holding half of either operand: a single SM
//         at 128 x 256 would need 96 bytes a cycle from L2, against the 64
//         it can take; the pair needs 64), two accumulators in tensor memory,
//         so a tile's epilogue runs under the next tile's products;
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
constexpr uint32_t kLoaders = 512;

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
  uint32_t bn, bq;     // rows of Q in a tile, and in a block's stage
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

template <bool kPair>
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap* map, uint32_t x, uint32_t y, uint32_t bar) {
  if constexpr (kPair)
    tma_load_2d_pair(dst, map, x, y, bar);
  else
    tma_load_2d(dst, map, x, y, bar);
}

template <bool kPair>
__device__ __forceinline__ void copy_operand(uint32_t dst, const CUtensorMap* map, bool mn, uint32_t row0, uint32_t k0,
                                             uint32_t rows, uint32_t bar) {
  if (!mn) {
    copy_box<kPair>(dst, map, k0, row0, bar);
  } else {
    for (uint32_t r = 0; r < rows; r += 64) copy_box<kPair>(dst + r * 128, map, row0 + r, k0, bar);
  }
}

// ---- filling a stage with plain loads -------------------------------------------------
//
// A stage is (128 + bn) rows of eight 16-byte units; a unit's 8 elements may
// start at any even address.  Aligned 16-byte loads cover it: a thread loads
// the aligned unit at or below its address, takes the next one from its
// neighbour in the row (the last of a row loads it), and shifts the 8
// elements out of the pair.  Nothing outside [lo, hi), the matrix's first and
// last byte, is touched: units whose aligned loads would cross them go element
// by element.

struct Operand {
  const uint16_t* p;
  uint64_t ld;
  uint32_t nrows, ncols;  // as stored
  uint32_t mn, row0;      // the tile's first matrix row
  uintptr_t lo, hi;
};

__device__ __forceinline__ Operand operand(const uint16_t* p, uint64_t ld, uint32_t mn, uint32_t rows, uint32_t k,
                                           uint32_t row0) {
  Operand o{p, ld, mn ? k : rows, mn ? rows : k, mn, row0, 0, 0};
  o.lo = reinterpret_cast<uintptr_t>(p);
  o.hi = o.lo + ((o.nrows - 1) * ld + o.ncols) * 2;
  return o;
}

// In flight: one unit of a thread.
struct Unit {
  uint4 a, b;
  uintptr_t at;    // address of the unit's first element
  int n;           // its elements inside the matrix, at most 8 (0 or less: none)
  uint32_t flags;  // 1: `a` was loaded, 2: `b` was loaded
};

__device__ __forceinline__ void unit_load(Unit& t, const Operand& o, uint32_t id, uint32_t k0) {
  const uint32_t line = id >> 3, u = id & 7u;
  const uint32_t row = o.mn ? k0 + (line & 63u) : o.row0 + line;
  const uint32_t col = (o.mn ? o.row0 + (line >> 6) * 64 : k0) + u * 8;
  t.a = t.b = make_uint4(0, 0, 0, 0);
  t.n = row < o.nrows ? int(o.ncols) - int(col) : -8;
  t.at = reinterpret_cast<uintptr_t>(o.p + row * o.ld + col);
  t.flags = 0;
  const uintptr_t q = t.at & ~uintptr_t(15);
  // Also loaded when only the unit before needs it.
  if (t.n > -8 && q >= o.lo && q + 16 <= o.hi) {
    t.a = *reinterpret_cast<const uint4*>(q);
    t.flags = 1;
  }
  if (u == 7 && t.n > 0 && (t.at & 15) != 0 && q + 32 <= o.hi) {
    t.b = *reinterpret_cast<const uint4*>(q + 16);
    t.flags |= 2;
  }
}

__device__ __forceinline__ void unit_store(Unit& t, uint32_t id, uint8_t* dst) {
  const uint32_t u = id & 7u;
  uint4 nb;
  nb.x = __shfl_down_sync(0xFFFFFFFFu, t.a.x, 1);
  nb.y = __shfl_down_sync(0xFFFFFFFFu, t.a.y, 1);
  nb.z = __shfl_down_sync(0xFFFFFFFFu, t.a.z, 1);
  nb.w = __shfl_down_sync(0xFFFFFFFFu, t.a.w, 1);
  const uint32_t nf = __shfl_down_sync(0xFFFFFFFFu, t.flags, 1);
  if (u != 7) {
    t.b = nb;
    if (nf & 1) t.flags |= 2;
  }
  const uint32_t mis = uint32_t(t.at & 15);
  const int n = t.n > 8 ? 8 : t.n;
  uint32_t w[4] = {0, 0, 0, 0};
  if (n > 0) {
    if ((t.flags & 1) && (mis + 2 * n <= 16 || (t.flags & 2))) {
      uint32_t s[8] = {t.a.x, t.a.y, t.a.z, t.a.w, t.b.x, t.b.y, t.b.z, t.b.w};
      if (mis & 8)
#pragma unroll
        for (int i = 0; i < 6; ++i) s[i] = s[i + 2];
      if (mis & 4)
#pragma unroll
        for (int i = 0; i < 5; ++i) s[i] = s[i + 1];
      const uint32_t shift = (mis & 2) * 8;
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(s[i], s[i + 1], shift);
      if (n < 8)
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] &= n >= 2 * i + 2 ? 0xFFFFFFFFu : (n == 2 * i + 1 ? 0xFFFFu : 0u);
    } else {
      const uint16_t* p = reinterpret_cast<const uint16_t*>(t.at);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) w[i >> 1] |= uint32_t(p[i]) << (16 * (i & 1));
    }
  }
  const uint32_t line = id >> 3;
  *reinterpret_cast<uint4*>(dst + line * 128 + ((u ^ (line & 7u)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
}

// kN units of a thread at once: their loads are in flight together.
template <int kN>
__device__ __forceinline__ void load_units(const Operand& o, uint8_t* dst, uint32_t first, uint32_t k0) {
  Unit t[kN];
#pragma unroll
  for (int j = 0; j < kN; ++j) unit_load(t[j], o, first + j * kLoaders, k0);
#pragma unroll
  for (int j = 0; j < kN; ++j) unit_store(t[j], first + j * kLoaders, dst);
}

__device__ __forceinline__ void load_stage(const Operand& p, const Operand& q, uint8_t* dst, uint32_t bn, uint32_t k0,
                                           uint32_t tid) {
  load_units<kLanes * 8 / kLoaders>(p, dst, tid, k0);
  const uint32_t units = bn * 8;
  uint32_t i = tid;
  for (; i + kLoaders < units; i += 2 * kLoaders) load_units<2>(q, dst + kPBytes, i, k0);
  if (i < units) load_units<1>(q, dst + kPBytes, i, k0);  // whole warps: units and kLoaders are multiples of 32
}

// ---- the roles, for one tile -------------------------------------------------------

// One thread (the copy engine) or kLoaders threads.  In a pair each block
// fills its own half of the stage; both halves count on the first block's
// barrier.  Returns false after a wait ran out.
template <bool kTma, bool kPair>
__device__ __forceinline__ bool fill_tile(const GemmArgs& a, const CUtensorMap* mp, const CUtensorMap* mq, Shared& s,
                                          uint8_t* stages, Ring& ring, uint32_t p0, uint32_t q0, uint32_t first,
                                          uint32_t last, uint32_t tid, uint32_t rank) {
  Operand op, oq;
  if constexpr (!kTma) {
    op = operand(a.p, a.ldp, a.p_mn, a.P, a.K, p0);
    oq = operand(a.q, a.ldq, a.q_mn, a.Q, a.K, q0);
  }
  for (uint32_t i = first; i < last; ++i) {
    bool ok = mbar_wait(addr_of(&s.empty[ring.slot]), ring.phase ^ 1, &s.abort);
    if constexpr (!kTma) ok = __all_sync(0xFFFFFFFFu, ok);
    if (!ok) return false;
    uint8_t* dst = stages + ring.slot * a.stage_bytes;
    uint32_t bar = addr_of(&s.full[ring.slot]);
    if constexpr (kTma) {
      if (!kPair || rank == 0) mbar_arrive_expect(bar, kPair ? 2 * a.stage_bytes : a.stage_bytes);
      if (kPair) bar = cluster_peer_address(bar, 0);
      copy_operand<kPair>(addr_of(dst), mp, a.p_mn, p0, i * kStep, kLanes, bar);
      copy_operand<kPair>(addr_of(dst) + kPBytes, mq, a.q_mn, q0, i * kStep, a.bq, bar);
    } else {
      load_stage(op, oq, dst, a.bq, i * kStep, tid);
      fence_async_shared();
      __syncwarp();
      if (tid % 32 == 0) {
        if (kPair)
          mbar_arrive_cluster(cluster_peer_address(bar, 0));
        else
          mbar_arrive(bar);
      }
    }
    ring.next(a.stages);
  }
  return true;
}

// One thread (of a pair's first block) issues the tile's products into `tmem`.
template <bool kPair>
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
      mma_f16<kPair>(tmem, dp + k * adv_p, dq + k * adv_q, a.idesc, i != first || k != 0);
    mma_commit<kPair>(addr_of(&s.empty[ring.slot]));
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

template <bool kTma, bool kPair>
__device__ __forceinline__ void setup(const GemmArgs& a, const CUtensorMap* mp, const CUtensorMap* mq, Shared& s,
                                      uint32_t warp) {
  if (threadIdx.x == 0) {
    for (uint32_t i = 0; i < a.stages; ++i) {
      mbar_init(addr_of(&s.full[i]), kTma ? 1 : (kPair ? 2 : 1) * (kLoaders / 32));
      mbar_init(addr_of(&s.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(addr_of(&s.acc_full[i]), 1);
      mbar_init(addr_of(&s.acc_empty[i]), 8);  // the epilogue warps of a pair
    }
    mbar_init(addr_of(&s.drain), 1);
    s.abort = 0;
    mbar_init_fence();
    if (kTma) prefetch_tensor_map(mp), prefetch_tensor_map(mq);
  }
  if (warp == 1) tmem_alloc<kPair>(addr_of(&s.tmem), a.tmem_columns);
  tmem_fence_before();
  __syncthreads();
  if (kPair) {  // the peer's barriers are ready before a copy counts on them
    cluster_arrive_release();
    cluster_wait();
  }
  tmem_fence_after();
}

// Every thread, after its role; kCluster: the cluster's blocks read or signal
// each other's memory, so none leaves before all are done.  When a wait ran
// out in any of them, the copies and the matrix instructions still in flight
// are waited for, again with a bound, before the memory is given up.  `ring`,
// `issued`: the copying thread's next stage and an upper bound of the stages
// it filled.
template <bool kTma, bool kPair>
__device__ __forceinline__ void finish_block(const GemmArgs& a, Shared& s, uint32_t warp, uint32_t lane, uint32_t rank,
                                             Ring ring, uint32_t issued) {
  tmem_fence_before();
  __syncthreads();
  cluster_arrive_release();
  cluster_wait();
  tmem_fence_after();
  uint32_t gave_up = s.abort;
  if (kPair) gave_up |= ld_cluster_u32(cluster_peer_address(addr_of(const_cast<uint32_t*>(&s.abort)), rank ^ 1));
  if (gave_up) {
    volatile uint32_t own = 0;
    if (kTma && threadIdx.x == 0 && (!kPair || rank == 0)) {
      for (uint32_t i = 0; i < issued && i < a.stages; ++i) {
        if (ring.slot == 0) ring.slot = a.stages, ring.phase ^= 1;
        --ring.slot;
        mbar_wait(addr_of(&s.full[ring.slot]), ring.phase, &own);
      }
    }
    if (warp == 1 && lane == 0 && (!kPair || rank == 0)) {
      mma_commit<kPair>(addr_of(&s.drain));
      mbar_wait(addr_of(&s.drain), 0, &own);
    }
    if (threadIdx.x == 0 && a.status) *a.status = uint32_t(ARX_ETIMEOUT) | (12u << 8);
  }
  if (kPair) {  // after the peer's abort word was read, and any drain
    __syncwarp();
    cluster_arrive_release();
    cluster_wait();
  } else {
    __syncthreads();
  }
  if (warp == 1) tmem_free<kPair>(s.tmem, a.tmem_columns);
}

template <bool kTma>
constexpr uint32_t kGemmThreads = kTma ? 192 : 192 + kLoaders;

// The same of 4 consecutive columns.
template <int D>
__device__ __forceinline__ void finish4(const GemmArgs& a, float (&v)[4], uint32_t row, uint32_t col) {
  uint16_t* out = a.out + row * a.ldout + col;
  const uint32_t n = col < a.P ? a.P - col : 0;
  const bool whole = a.vec && n >= 4;
#pragma unroll
  for (uint32_t k = 0; k < 4; ++k)
    if (a.bias && k < n) v[k] += load_param(a.bias, a.wdtype, col + k);
  if (a.z) {
    uint16_t* z = a.z + row * a.ldz + col;
    if (whole) {
      st_global(reinterpret_cast<uint2*>(z), make_uint2(Elem<D>::round2(v[0], v[1]), Elem<D>::round2(v[2], v[3])));
    } else {
#pragma unroll
      for (uint32_t k = 0; k < 4; ++k)
        if (k < n) z[k] = Elem<D>::round(v[k]);
    }
  }
  activate<4>(v, a.act);
  if (a.residual)
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k)
      if (k < n) v[k] += Elem<D>::widen(a.residual[row * a.ldresidual + col + k]);
  if (whole) {
    st_global(reinterpret_cast<uint2*>(out), make_uint2(Elem<D>::round2(v[0], v[1]), Elem<D>::round2(v[2], v[3])));
  } else {
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k)
      if (k < n) out[k] = Elem<D>::round(v[k]);
  }
}

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
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x & 31, rank = cluster_ctarank();
  setup<kTma, true>(a, &mp, &mq, s, warp);
  dependent_launch_prologue();
  const uint32_t tiles = a.tiles_p * a.tiles_q, first_tile = blockIdx.x / 2, step = gridDim.x / 2;

  Ring ring;
  uint32_t issued = 0;
  if (kTma ? threadIdx.x == 0 : warp >= 6) {
    for (uint32_t t = first_tile; t < tiles; t += step) {
      uint32_t tp, tq;
      tile_at(a, t, tp, tq);
      issued = a.stages;
      if (!fill_tile<kTma, true>(a, &mp, &mq, s, stages, ring, (2 * tp + rank) * kLanes, tq * a.bn + rank * a.bq, 0,
                                 a.steps, threadIdx.x - (kTma ? 0 : 192), rank))
        break;
    }
  } else if (warp == 1 && lane == 0 && rank == 0 && a.steps > 0) {
    uint32_t n = 0;
    for (uint32_t t = first_tile; t < tiles; t += step, ++n) {
      const uint32_t b = n & 1, use = n >> 1;
      if (!mbar_wait(addr_of(&s.acc_empty[b]), (use & 1) ^ 1, &s.abort)) break;
      tmem_fence_after();
      if (!multiply_tile<true>(a, s, addr_of(stages), ring, s.tmem + b * 256, 0, a.steps)) break;
      mma_commit<true>(addr_of(&s.acc_full[b]));
    }
  } else if (warp >= 2 && warp < 6) {
    const uint32_t quarter = warp & 3;  // the accumulator lanes this warp may read
    uint32_t n = 0;
    for (uint32_t t = first_tile; t < tiles; t += step, ++n) {
      uint32_t tp, tq;
      tile_at(a, t, tp, tq);
      const uint32_t b = n & 1, use = n >> 1;
      if (a.steps > 0) {
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(addr_of(&s.acc_full[b]), use & 1, &s.abort))) break;
        tmem_fence_after();
      }
      const uint32_t row = (2 * tp + rank) * kLanes + quarter * 32 + lane, col0 = tq * a.bn;
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
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(cluster_peer_address(addr_of(&s.acc_empty[b]), 0));
    }
  }
  __syncwarp();
  finish_block<kTma, true>(a, s, warp, lane, rank, ring, issued);
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
  setup<kTma, false>(a, &mp, &mq, s, warp);
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
    fill_tile<kTma, false>(a, &mp, &mq, s, stages, ring, p0, q0, first, last, threadIdx.x - (kTma ? 0 : 192), 0);
  } else if (warp == 1 && lane == 0 && first < last) {
    if (multiply_tile<false>(a, s, addr_of(stages), ring, s.tmem, first, last))
      mma_commit<false>(addr_of(&s.acc_full[0]));
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
  // shared out over the cluster's blocks in groups of four lanes; each is the
  // sum of the partials in block order.
  const uint32_t nq = a.Q - q0 < a.bn ? a.Q - q0 : a.bn;
  const uint32_t groups = nq * (kLanes / 4);
  const uint32_t per = (groups + a.split - 1) / a.split;
  const uint32_t end = (rank + 1) * per < groups ? (rank + 1) * per : groups;
  const uint32_t at = addr_of(part);
  for (uint32_t i = rank * per + threadIdx.x; i < end; i += kGemmThreads<kTma>) {
    const uint32_t j = p0 + (i * 4 & (kLanes - 1)), row = q0 + i / (kLanes / 4);
    float4 in[8];
#pragma unroll
    for (uint32_t r = 0; r < 8; ++r)
      if (r < a.split) in[r] = ld_cluster_f32x4(cluster_peer_address(at + i * 16, r));
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (uint32_t r = 0; r < 8; ++r)
      if (r < a.split) v[0] += in[r].x, v[1] += in[r].y, v[2] += in[r].z, v[3] += in[r].w;
    finish4<D>(a, v, row, j);
  }
  finish_block<kTma, false>(a, s, warp, lane, rank, ring, last - first);
}

// ---- one to four rows ------------------------------------------------------------------
//
// out[m][j] = sum_k x[m][k] w[j][k]: w is read once, which bounds the kernel,
// at 2 M operations to an element.  A warp (or `split` warps of a block) takes
// a feature j; its lanes take 16-byte units of the row, kBatch of them in
// flight, and x comes from L1.  The lanes' sums meet in a butterfly and the
// split warps' in warp order.  kV = 1: rows off 16 bytes, element by element.

constexpr uint32_t kDotRows = 4;
constexpr uint32_t kDotThreads = 256;
constexpr int kDotBatch = 8;

template <int D, int kM, int kV>
__global__ void __launch_bounds__(kDotThreads) dot_kernel(const __grid_constant__ GemmArgs a) {
  __shared__ float part[kDotThreads / 32][kM];
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const uint32_t per = kDotThreads / 32 / a.split;             // features of a block
  const uint32_t j = blockIdx.x * per + warp / a.split, share = warp % a.split;
  // A hint only (as in the reduce kernels): the weights' way to L2 starts
  // while the stream's previous kernel, whose output x may be, still runs.
  if (kV == 8 && share == 0 && lane == 0 && j < a.Q && a.K > 0) prefetch_l2_bulk(a.q + j * a.ldq, a.K * 2);
  dependent_launch_prologue();
  float acc[kM] = {};
  if (j < a.Q) {
    const uint16_t* w = a.q + j * a.ldq;
    const uint32_t units = a.K / kV, step = 32 * a.split;
    for (uint32_t u0 = share * 32 + lane; u0 < units; u0 += kDotBatch * step) {
      Pack<D, kV> wv[kDotBatch];
#pragma unroll
      for (int b = 0; b < kDotBatch; ++b)
        if (u0 + b * step < units)
          wv[b].load(w + size_t(u0 + b * step) * kV);
        else
          wv[b].zero();
#pragma unroll
      for (int b = 0; b < kDotBatch; ++b) {
        if (u0 + b * step >= units) break;
        float f[kV];
        wv[b].get(f);
#pragma unroll
        for (int m = 0; m < kM; ++m) {
          float x[kV];
          load_params<kV>(a.p + m * a.ldp, D, size_t(u0 + b * step) * kV, x);
#pragma unroll
          for (int k = 0; k < kV; ++k) acc[m] = fmaf(f[k], x[k], acc[m]);
        }
      }
    }
  }
#pragma unroll
  for (int m = 0; m < kM; ++m) acc[m] = warp_sum(acc[m]);
  if (a.split > 1) {
    if (lane == 0)
#pragma unroll
      for (int m = 0; m < kM; ++m) part[warp][m] = acc[m];
    __syncthreads();
    if (share == 0)
      for (uint32_t r = 1; r < a.split; ++r)
#pragma unroll
        for (int m = 0; m < kM; ++m) acc[m] += part[warp + r][m];
  }
  if (share != 0 || j >= a.Q) return;
#pragma unroll
  for (int m = 0; m < kM; ++m)
    if (lane == uint32_t(m)) {
      float f[1] = {acc[m]};
      if (a.bias) f[0] += load_param(a.bias, a.wdtype, j);
      if (a.z) a.z[m * a.ldz + j] = Elem<D>::round(f[0]);
      activate<1>(f, a.act);
      if (a.residual) f[0] += Elem<D>::widen(a.residual[m * a.ldresidual + j]);
      a.out[m * a.ldout + j] = Elem<D>::round(f[0]);
    }
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

// Launch with clusters of `cluster` blocks.
template <auto kKernel>
cudaError_t launch_cluster(uint32_t blocks, uint32_t threads, uint32_t cluster, uint32_t smem, cudaStream_t st,
                           const GemmArgs& a, const CUtensorMap& mp, const CUtensorMap& mq) {
  cudaError_t e = allow_smem<kKernel>();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kKernel, a, mp, mq);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// A persistent grid: as many pairs as the device holds at once (two blocks to
// a pair, one block to an SM), or fewer tiles.
template <int D, bool kTma>
cudaError_t launch_wide(const GemmArgs& a, const CUtensorMap& mp, const CUtensorMap& mq, int sms, cudaStream_t st) {
  const uint32_t tiles = a.tiles_p * a.tiles_q, pairs = uint32_t(sms) / 2;
  return launch_cluster<gemm_wide_kernel<D, kTma>>(2 * (tiles < pairs ? tiles : pairs), kGemmThreads<kTma>, 2,
                                                   kStageBudget + 1024, st, a, mp, mq);
}

template <int D, bool kTma>
cudaError_t launch_split(const GemmArgs& a, const CUtensorMap& mp, const CUtensorMap& mq, cudaStream_t st) {
  return launch_cluster<gemm_split_kernel<D, kTma>>(a.tiles_p * a.tiles_q * a.split, kGemmThreads<kTma>, a.split,
                                                    kStageBudget + 1024, st, a, mp, mq);
}

uint32_t ceil_div(uint64_t a, uint64_t b) { return uint32_t((a + b - 1) / b); }

template <int D, int kV>
cudaError_t launch_dot(const GemmArgs& a, cudaStream_t st) {
  const dim3 grid(ceil_div(a.Q, kDotThreads / 32 / a.split));
  switch (a.P) {
    case 1: return launch_op(dot_kernel<D, 1, kV>, grid, kDotThreads, 0, st, a);
    case 2: return launch_op(dot_kernel<D, 2, kV>, grid, kDotThreads, 0, st, a);
    case 3: return launch_op(dot_kernel<D, 3, kV>, grid, kDotThreads, 0, st, a);
    default: return launch_op(dot_kernel<D, 4, kV>, grid, kDotThreads, 0, st, a);
  }
}

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

  const bool bf16 = c.dtype == ARX_BF16;
  if (c.rows <= kDotRows && !c.p_mn && !c.q_mn) {
    a.p = static_cast<const uint16_t*>(c.p), a.q = static_cast<const uint16_t*>(c.q);
    a.ldp = c.ldp, a.ldq = c.ldq;
    a.P = uint32_t(c.rows), a.Q = uint32_t(c.cols);
    const bool units = a.K % 8 == 0 && copyable(a.p, a.ldp, a.P) && copyable(a.q, a.ldq, a.Q);
    // Warps for about 16 to an SM, while each keeps 256 elements or more.
    a.split = 1;
    while (a.split < 8 && uint64_t(a.Q) * a.split < 2432 && a.K / a.split > 512) a.split *= 2;
    if (bf16) return units ? launch_dot<ARX_BF16, 8>(a, st) : launch_dot<ARX_BF16, 1>(a, st);
    return units ? launch_dot<ARX_F16, 8>(a, st) : launch_dot<ARX_F16, 1>(a, st);
  }

  // Wide tiles when they occupy most of the SMs, else the split form.
  const bool wide = uint64_t(ceil_div(c.rows, kLanes)) * ceil_div(c.cols, 256) >= 100;
  const auto *cp = static_cast<const uint16_t*>(c.p), *cq = static_cast<const uint16_t*>(c.q);
  if (wide) {
    a.p = cp, a.q = cq, a.ldp = c.ldp, a.ldq = c.ldq, a.p_mn = c.p_mn, a.q_mn = c.q_mn;
    a.P = uint32_t(c.rows), a.Q = uint32_t(c.cols);
    a.bn = 256;
    a.bq = a.bn / 2;
    a.split = 1;
    a.tmem_columns = 512;
  } else {
    a.p = cq, a.q = cp, a.ldp = c.ldq, a.ldq = c.ldp, a.p_mn = c.q_mn, a.q_mn = c.p_mn;
    a.P = uint32_t(c.cols), a.Q = uint32_t(c.rows);
    a.bn = a.q_mn ? 64 : 16;
    while (a.bn < a.Q && a.bn < 256) a.bn *= 2;
    a.bq = a.bn;
    a.tmem_columns = a.bn < 32 ? 32 : a.bn;
    const uint32_t tiles = ceil_div(a.P, kLanes) * ceil_div(a.Q, a.bn);
    a.split = 1;
    while (a.split < 8 && 2 * a.split * tiles <= uint32_t(sms) && 2 * a.split <= a.steps) a.split *= 2;
  }
  const uint32_t lanes = wide ? 2 * kLanes : kLanes;
  a.tiles_p = ceil_div(a.P, lanes);
  a.tiles_q = ceil_div(a.Q, a.bn);
  a.stage_bytes = kPBytes + a.bq * 128;
  a.stages = kStageBudget / a.stage_bytes;
  if (a.stages > kMaxStages) a.stages = kMaxStages;
  a.idesc = mma_descriptor(c.dtype == ARX_BF16, a.p_mn, a.q_mn, lanes, a.bn);

  const uint64_t p_rows = a.p_mn ? a.K : a.P, q_rows = a.q_mn ? a.K : a.Q;
  const bool tma = a.K > 0 && copyable(a.p, a.ldp, p_rows) && copyable(a.q, a.ldq, q_rows);
  CUtensorMap mp{}, mq{};
  if (tma) {
    err = encode(&mp, a.p, a.ldp, p_rows, a.p_mn ? a.P : a.K, a.p_mn ? 64 : kLanes, bf16);
    if (err != cudaSuccess) return err;
    err = encode(&mq, a.q, a.ldq, q_rows, a.q_mn ? a.Q : a.K, a.q_mn ? 64 : a.bq, bf16);
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
