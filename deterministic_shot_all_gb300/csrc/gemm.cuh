// Parts of the matrix products on the tensor cores that their kernels share
// (linear.cu, gated.cu): the ring of stages and who fills it, the matrix
// instructions, the order of tiles, what a block does when a wait ran out, and the
// maps of the copy engine.
#pragma once

#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <type_traits>

#include "arx_internal.h"
#include "arx_rows.cuh"
#include "forms.h"
#include "ops_launch.h"
#include "spans.h"
#include "tensor_core.cuh"

namespace arx {
namespace {

constexpr uint32_t kPBytes = kLanes * 128;   // P's part of a stage
constexpr uint32_t kMaxStages = 12;
// Shared memory of a block's stages.  One wide block, or two split blocks of
// up to 128 accumulator columns, fit an SM at a time, so the blocks on an SM
// never want more tensor memory than it has (a block that waited for columns
// while its cluster waited for it could wait forever).  Of blocks with loading
// threads one fits, by its 704 threads' registers, and two to four stages took
// the same time; a wide one asks for more than it uses (kAloneShared), so that
// no split block fits beside its 512 columns however few registers it takes.
constexpr uint32_t kStageBudget = 196608, kSplitBudget = 98304, kLoadedBudget = 98304;
constexpr uint32_t kAloneShared = 155648;
// The split form's stages of 16 + 2, 4, 8 and 16 KB; an SM has 228 KB, 1 KB of
// it goes with every block.
constexpr uint32_t split_shared(uint32_t bn) { return 1024 + kSplitBudget / (kPBytes + bn * 128) * (kPBytes + bn * 128); }
static_assert(kAloneShared + split_shared(16) + 2048 > 233472 && kAloneShared + split_shared(32) + 2048 > 233472 &&
              kAloneShared + split_shared(64) + 2048 > 233472 && kAloneShared + split_shared(128) + 2048 > 233472);
constexpr uint32_t kStagedBytes = 32 * 33 * 4;  // of an epilogue warp of the wide form
constexpr uint32_t kMostShared = kStageBudget + 1024 + 8 * kStagedBytes;
constexpr uint32_t kLoaders = 512;

struct GemmArgs {
  const uint16_t *p, *q;
  uint64_t ldp, ldq;
  uint32_t P, Q, K;
  uint32_t p_mn, q_mn;
  uint32_t p_copy, q_copy;  // the copy engine brings the operand in, not threads
  uint32_t p_layout, q_layout;
  uint16_t *out, *z;
  const void* bias;
  const uint16_t* residual;
  uint64_t ldout, ldz, ldresidual;
  uint32_t* status;
  uint32_t wait_ns;    // limit of a wait
  int act, wdtype;
  uint32_t bn, bq;     // rows of Q under one accumulator, and a block's share of them in a stage
  uint32_t stages, stage_bytes;
  uint32_t steps;      // stages' worth of contraction: ceil(K / 64), of two pairs of operands both
  uint32_t first_steps;  // of the first pair, where there are two
  uint32_t split;      // blocks of a cluster that share a tile's contraction
  uint32_t whole, pieces;  // wide form: tiles that are one piece, and pieces in all
  uint32_t tiles_p, tiles_q;
  uint32_t tiles_first;  // of the first of two stacked products
  uint16_t* out2;        // the second's output
  uint64_t ldout2;
  uint32_t idesc, tmem_columns;
  uint32_t quads, octets;  // out, z and residual allow accesses of 4 elements; of 8, bias and width too
};

struct Shared {
  uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], drain;
  uint32_t fills[1 + kLoaders / 32];  // of the copying thread and of each loading warp, once its role ends
  uint32_t tmem;
  volatile Waits waits;
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

// Layouts of an operand in memory.
enum Layout : uint32_t {
  kKMajor,    // matrix rows: one box of 64 contraction elements
  kMnMajor,   // contraction rows: a box for every 64 matrix rows
  kMnBlocks,  // the same with whole blocks of 64: one box over the blocks of a map (64, k, block);
              // dz^T x of 8192 x 4096 over 8185 tokens: 309 us, with a box to each block 361
};

template <bool kPair>
__device__ __forceinline__ void copy_operand(uint32_t dst, const CUtensorMap* map, uint32_t layout, uint32_t row0,
                                             uint32_t k0, uint32_t rows, uint32_t bar) {
  if (layout == kKMajor) {
    copy_box<kPair>(dst, map, k0, row0, bar);
  } else if (layout == kMnBlocks) {
    tma_load_3d<kPair>(dst, map, k0, row0 / 64, bar);
  } else {
    for (uint32_t r = 0; r < rows; r += 64) copy_box<kPair>(dst + r * 128, map, row0 + r, k0, bar);
  }
}

// ---- the roles, for one tile -------------------------------------------------------

// A second product in the same launch (the backward pass of a gated block).
//  kSum    a second pair of operands, whose product joins the first's in one sum:
//          the contraction runs over the first pair, then over the second.
//  kStack  a second operand in the place of the call's p, with an output of its
//          own: its tiles follow the first's.
enum Extra : int { kNone, kSum, kStack };
template <int kExtra>
struct SecondMaps {};
template <>
struct SecondMaps<kSum> {
  CUtensorMap p, q;
};
template <>
struct SecondMaps<kStack> {
  CUtensorMap in, out;  // the operand (P of a wide tile, Q of a split one), the output
};

struct Output {
  uint16_t* p;
  uint64_t ld;
};

// Is tile t of the stacked dimension the second product's?  t counts from its
// own product's first then.
template <int kExtra>
__device__ __forceinline__ bool second_product(const GemmArgs& a, uint32_t& t) {
  if (kExtra != kStack || t < a.tiles_first) return false;
  t -= a.tiles_first;
  return true;
}
template <int kExtra>
__device__ __forceinline__ Output output_of(const GemmArgs& a, bool second) {
  if (kExtra == kStack && second) return {a.out2, a.ldout2};
  return {a.out, a.ldout};
}

// Bytes that the copy engine brings to a block's stage for `subs` accumulators.
__device__ __forceinline__ uint32_t copied_bytes(const GemmArgs& a, uint32_t subs) {
  return (a.p_copy ? kPBytes : 0) + (a.q_copy ? subs * a.bq * 128 : 0);
}

// One thread: the operands that the copy engine can address.  In a pair each
// block fills its own half of the stage; both halves count on the first
// block's barrier.  Returns the stages filled, fewer than last - first after a
// wait ran out.
template <bool kPair, uint32_t kSubs, int kExtra>
__device__ __forceinline__ uint32_t copy_tile(const GemmArgs& a, const CUtensorMap* mp, const CUtensorMap* mq,
                                              const SecondMaps<kExtra>* m2, Shared& s, uint8_t* stages, Ring& ring,
                                              uint32_t p0, uint32_t q0, uint32_t first, uint32_t last, uint32_t rank) {
  const uint32_t bytes = copied_bytes(a, kSubs);
  for (uint32_t i = first; i < last; ++i) {
    if (!mbar_wait(addr_of(&s.empty[ring.slot]), ring.phase ^ 1, &s.waits)) return i - first;
    uint8_t* dst = stages + ring.slot * a.stage_bytes;
    uint32_t bar = addr_of(&s.full[ring.slot]);
    if (!kPair || rank == 0) mbar_arrive_expect(bar, kPair ? 2 * bytes : bytes);
    if (kPair) bar = cluster_peer_address(bar, 0);
    const CUtensorMap *p = mp, *q = mq;
    uint32_t k0 = i * kStep;
    if constexpr (kExtra == kSum)
      if (i >= a.first_steps) p = &m2->p, q = &m2->q, k0 = (i - a.first_steps) * kStep;
    if (a.p_copy) copy_operand<kPair>(addr_of(dst), p, a.p_layout, p0, k0, kLanes, bar);
    if (a.q_copy)
#pragma unroll
      for (uint32_t j = 0; j < kSubs; ++j)
        copy_operand<kPair>(addr_of(dst) + kPBytes + j * a.bq * 128, q, a.q_layout, q0 + j * a.bn, k0, a.bq, bar);
    ring.next(a.stages);
  }
  return last - first;
}

// One thread (of a pair's first block) issues the tile's products into `tmem`.
template <bool kPair, uint32_t kSubs, bool k8 = false>  // k8: e4m3 operands
__device__ __forceinline__ bool multiply_tile(const GemmArgs& a, Shared& s, uint32_t stages, Ring& ring, uint32_t tmem,
                                              uint32_t first, uint32_t last) {
  // A contraction step of 16 (of 8-bit operands 32) is 32 bytes along a K-major
  // row, 16 rows of an MN-major tile; in the descriptors' units of 16 bytes.
  const uint32_t adv_p = a.p_mn ? 128 : 2, adv_q = a.q_mn ? 128 : 2;
  for (uint32_t i = first; i < last; ++i) {
    if (!mbar_wait(addr_of(&s.full[ring.slot]), ring.phase, &s.waits)) return false;
    tmem_fence_after();
    const uint32_t base = stages + ring.slot * a.stage_bytes;
    const uint64_t dp = operand_descriptor(base, kStep * 128), dq = operand_descriptor(base + kPBytes, kStep * 128);
#pragma unroll
    for (uint32_t k = 0; k < kStep / 16; ++k) {
      const bool sum = i != first || k != 0;
      if constexpr (k8) {
        mma_f8<kPair>(tmem, dp + k * adv_p, dq + k * adv_q, a.idesc, sum);
        if (kSubs == 2) mma_f8<kPair>(tmem + 256, dp + k * adv_p, dq + a.bq * 8 + k * adv_q, a.idesc, sum);
      } else {
        mma_f16<kPair>(tmem, dp + k * adv_p, dq + k * adv_q, a.idesc, sum);
        if (kSubs == 2) mma_f16<kPair>(tmem + 256, dp + k * adv_p, dq + a.bq * 8 + k * adv_q, a.idesc, sum);
      }
    }
    mma_commit<kPair>(addr_of(&s.empty[ring.slot]));
    ring.next(a.stages);
  }
  return true;
}

// As load_ahead16.
__device__ __forceinline__ uint2 load_ahead8(const void* p, bool on) {
  uint2 v;
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %3, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\t"
      "@q ld.global.v2.b32 {%0, %1}, [%2];\n\t}"
      : "=&r"(v.x), "=&r"(v.y) : "l"(p), "r"(uint32_t(on)) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t load_ahead4(const void* p, bool on) {
  uint32_t v;
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\tmov.b32 %0, 0;\n\t@q ld.global.b32 %0, [%1];\n\t}"
               : "=&r"(v) : "l"(p), "r"(uint32_t(on)) : "memory");
  return v;
}
__device__ __forceinline__ uint16_t load_ahead2(const void* p, bool on) {
  uint16_t v;
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\tmov.b16 %0, 0;\n\t@q ld.global.b16 %0, [%1];\n\t}"
               : "=&h"(v) : "l"(p), "r"(uint32_t(on)) : "memory");
  return v;
}

// Rows on 16 bytes (and operands by the copy engine: the threads that load
// others leave too few registers): a warp's 32 rows by 32 columns go to shared
// memory as the copy engine's box (64-byte rows, its 64-byte swizzle) and from
// there to the matrix, clipped at its edges.  A warp has two boxes, used in
// turn.  (Each lane storing its own row touched 32 lines with every access:
// backward products of 200 tokens, 4096 x 4096: 41.7 us against 35.9.)
struct Boxes {
  uint32_t addr, turn;
};

template <int D>
__device__ __forceinline__ void store_box(const CUtensorMap* map, const float (&v)[32], uint32_t row0, uint32_t col,
                                          Boxes& boxes, uint32_t lane) {
  const uint32_t box = boxes.addr + boxes.turn * 2048;
  boxes.turn ^= 1;
  if (lane == 0) bulk_wait_read<1>();  // the box's last store has read it
  __syncwarp();
#pragma unroll
  for (uint32_t u = 0; u < 4; ++u) {
    uint32_t w[4];
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) w[i] = Elem<D>::round2(v[8 * u + 2 * i], v[8 * u + 2 * i + 1]);
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                 :: "r"(box + lane * 64 + ((u ^ (lane >> 1 & 3u)) << 4)), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                 : "memory");
  }
  fence_async_shared();
  __syncwarp();
  if (lane == 0) tma_store_2d(map, col, row0, box);
}

// Warps: the copying one, the multiplying one, the epilogue's -- eight (two to
// a quarter of the lanes, halving the columns), four beside loading threads --
// and the loading threads.
template <bool kTma>
constexpr uint32_t kEpilogueWarps = kTma ? 8 : 4;
template <bool kTma>
constexpr uint32_t kFirstLoader = (2 + kEpilogueWarps<kTma>) * 32;
template <bool kTma>
constexpr uint32_t kGemmThreads = kFirstLoader<kTma> + (kTma ? 0 : kLoaders);

template <bool kTma, bool kPair>
__device__ __forceinline__ void setup(const GemmArgs& a, const CUtensorMap* mp, const CUtensorMap* mq, Shared& s,
                                      uint32_t warp) {
  if (threadIdx.x == 0) {
    for (uint32_t i = 0; i < a.stages; ++i) {
      mbar_init(addr_of(&s.full[i]), kTma ? 1 : (a.p_copy | a.q_copy) + (kPair ? 2 : 1) * (kLoaders / 32));
      mbar_init(addr_of(&s.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(addr_of(&s.acc_full[i]), 1);
      mbar_init(addr_of(&s.acc_empty[i]), 2 * kEpilogueWarps<kTma>);  // of a pair
    }
    mbar_init(addr_of(&s.drain), 1);
    s.waits.limit_ns = a.wait_ns, s.waits.abort = 0;
    mbar_init_fence();
    if (a.p_copy) prefetch_tensor_map(mp);
    if (a.q_copy) prefetch_tensor_map(mq);
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

// Tile order: bands of 8 row tiles, down the band first, so that the blocks
// at work at one time share operands in L2.
__device__ __forceinline__ void tile_at(const GemmArgs& a, uint32_t t, uint32_t& tp, uint32_t& tq) {
  const uint32_t band = 8u * a.tiles_q, b = t / band, in = t - b * band;
  const uint32_t rows = a.tiles_p - 8u * b < 8u ? a.tiles_p - 8u * b : 8u;
  tq = in / rows;
  tp = 8u * b + (in - tq * rows);
}

// The kernel's work in order.  Two accumulators to a tile (kSubs == 2): where
// the tiles past the last whole round of the grid would leave half of it or
// more without one, each of them is two pieces of one accumulator.
struct Piece {
  uint32_t tp, q0, subs;
};
template <uint32_t kSubs>
__device__ __forceinline__ Piece piece_at(const GemmArgs& a, uint32_t t) {
  Piece w{0, 0, kSubs};
  uint32_t tq, sub = 0;
  if (kSubs == 2 && t >= a.whole) {
    sub = (t - a.whole) & 1;
    w.subs = 1;
    t = a.whole + (t - a.whole) / 2;
  }
  tile_at(a, t, w.tp, tq);
  w.q0 = (tq * kSubs + sub) * a.bn;
  return w;
}

// A writer's fills, at the end of its role (see drain_block).
template <bool kTma>
__device__ __forceinline__ void note_fills(Shared& s, uint32_t fills, bool copies, uint32_t warp, uint32_t lane) {
  if (copies)
    s.fills[0] = fills;
  else if (!kTma && lane == 0)
    s.fills[1 + warp - kFirstLoader<kTma> / 32] = fills;
}

// After a wait ran out and every role (of a pair: of both blocks) has ended,
// nothing new is issued, but copies and matrix instructions may be in flight:
// they are waited for, with a bound, before memory is given up.  Of a pair, the
// first block does it, on whose barriers both blocks' copies count.
//
// One of a stage's writers -- the copying thread, in a pair the other block's
// too, the loading warps -- may have filled it where another gave up before, so
// that the stage's phase would never complete.  The writers' fills say which:
// what the missing ones would have announced and arrived with is made up for,
// and the phase completes exactly when the copies that were issued have landed.
// A writer fills a stage once its fill before, `stages` ago, was consumed: only
// the last `stages` of the writer that came furthest can be open.
// (Not inlined: the loading threads have no registers to spare.)
template <bool kTma, bool kPair, uint32_t kSubs>
__device__ __noinline__ void drain_block(const GemmArgs& a, Shared& s) {
  constexpr uint32_t kBlocks = kPair ? 2 : 1, kWriters = kTma ? 1 : 1 + kLoaders / 32;
  const uint32_t copies = a.p_copy | a.q_copy;
  volatile Waits own{kWaitNs, 0};
  if (threadIdx.x == 0) {
    const auto fills = [&](uint32_t block, uint32_t writer) {
      const uint32_t at = addr_of(&s.fills[writer]);
      return ld_cluster_u32(cluster_peer_address(at, kPair ? block : cluster_ctarank()));
    };
    uint32_t most = 0;
    for (uint32_t b = 0; b < kBlocks; ++b)
      for (uint32_t w = copies ? 0 : 1; w < kWriters; ++w) most = fills(b, w) > most ? fills(b, w) : most;
    for (uint32_t f = most > a.stages ? most - a.stages : 0; f < most; ++f) {
      const uint32_t bar = addr_of(&s.full[f % a.stages]);
      if (copies) {
        const bool mine = fills(0, 0) > f, peer = kPair && fills(1, 0) > f;
        const uint32_t piece = blockIdx.x / 2 + f / a.steps * (gridDim.x / 2);  // of a pair
        const uint32_t bytes = copied_bytes(a, kSubs == 2 ? piece_at<kSubs>(a, piece).subs : 1);
        if (mine) {
          if (kPair && !peer) mbar_complete_tx(bar, bytes);  // announced for both
        } else if (peer) {
          mbar_arrive_expect(bar, bytes);
        } else {
          mbar_arrive(bar);
        }
      }
      for (uint32_t b = 0; b < kBlocks; ++b)
        for (uint32_t w = 1; w < kWriters; ++w)
          if (fills(b, w) <= f) mbar_arrive(bar);
      mbar_wait(bar, f / a.stages & 1, &own);
    }
  }
  if (threadIdx.x == 32) {  // issued them
    mma_commit_own<kPair>(addr_of(&s.drain));
    mbar_wait(addr_of(&s.drain), 0, &own);
  }
}

// Every thread, after its role.  A cluster's blocks read or signal each
// other's memory, so none leaves before all are done.  (A block of the split
// form drains before it joins the others.)
template <bool kTma, bool kPair, uint32_t kSubs>
__device__ __forceinline__ void finish_block(const GemmArgs& a, Shared& s, uint32_t warp, uint32_t rank) {
  tmem_fence_before();
  __syncthreads();
  cluster_arrive_release();
  cluster_wait();
  tmem_fence_after();
  uint32_t gave_up = s.waits.abort;
  if (kPair) gave_up |= ld_cluster_u32(cluster_peer_address(addr_of(const_cast<uint32_t*>(&s.waits.abort)), rank ^ 1));
  if (gave_up) {
    if (kPair && rank == 0) drain_block<kTma, true, kSubs>(a, s);
    if (threadIdx.x == 0 && a.status) *a.status = uint32_t(ARX_ETIMEOUT) | (12u << 8);
  }
  if (kPair) {  // after the peer's words were read, and any drain
    __syncwarp();
    cluster_arrive_release();
    cluster_wait();
  } else {
    __syncthreads();
  }
  if (warp == 1) tmem_free<kPair>(s.tmem, a.tmem_columns);
}

// ---- host side ---------------------------------------------------------------------

// cuTensorMapEncodeTiled, looked up once through the runtime (the library
// links no driver library).
inline PFN_cuTensorMapEncodeTiled_v12000 encode_function(cudaError_t* err) {
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

// Map of an operand of `rows` by `k`, for tiles of `tile` rows by 64 of the
// contraction.
inline cudaError_t encode(CUtensorMap* m, uint32_t* layout, const uint16_t* base, uint64_t ld, uint32_t rows, uint32_t k,
                   bool mn, uint32_t tile, bool bf16) {
  cudaError_t err = cudaSuccess;
  auto f = encode_function(&err);
  if (!f) return err;
  *layout = !mn ? kKMajor : rows % 64 == 0 ? kMnBlocks : kMnMajor;
  const uint64_t inner = mn ? rows : k, outer = mn ? k : rows;
  const cuuint64_t pitch = (outer > 1 ? ld : (inner + 7) / 8 * 8) * 2;
  const cuuint64_t dims[3] = {*layout == kMnBlocks ? 64 : inner, outer, rows / 64}, strides[2] = {pitch, 128};
  const cuuint32_t box[3] = {64, mn ? 64 : tile, tile / 64}, el[3] = {1, 1, 1};
  const CUresult r = f(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                       *layout == kMnBlocks ? 3 : 2, const_cast<uint16_t*>(base), dims, strides, box, el,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Map of an output, for boxes of 32 rows by 32 columns (in store_box's swizzle) or
// 16 (without).
inline cudaError_t encode_output(CUtensorMap* m, uint16_t* base, uint64_t ld, uint32_t rows, uint32_t cols, bool bf16,
                                 uint32_t box_columns = 32) {
  cudaError_t err = cudaSuccess;
  auto f = encode_function(&err);
  if (!f) return err;
  const cuuint64_t dims[2] = {cols, rows}, strides[1] = {(rows > 1 ? ld : cols) * 2};
  const cuuint32_t box[2] = {box_columns, 32}, el[2] = {1, 1};
  const CUresult r = f(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, base, dims,
                       strides, box, el, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       box_columns == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_NONE,
                       CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

inline bool copyable(const uint16_t* p, uint64_t ld, uint64_t nrows) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (nrows <= 1 || ld % 8 == 0);
}

// Launch with clusters of `cluster` blocks.
template <auto kKernel, typename... A>
cudaError_t launch_cluster(uint32_t blocks, uint32_t threads, uint32_t cluster, uint32_t smem, cudaStream_t st,
                           const A&... args) {
  cudaError_t e = allow_dynamic_smem<kKernel>(kMostShared);
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
  e = cudaLaunchKernelEx(&cfg, kKernel, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace
}  // namespace arx
