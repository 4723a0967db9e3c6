// Matrix products on the tensor cores, with the epilogue of arx_linear.
//
// out[i][j] = act(sum_k P(i, k) Q(j, k) + bias[j]) + residual[i][j], 16-bit
// operands, fp32 accumulation in tensor memory.  The three products of a
// linear layer are this one with other operand layouts: x w^T (both operands
// K-major), dz w (w MN-major) and dz^T x (both MN-major); the copy engine
// brings 64-element boxes into 128-byte-swizzled shared memory either way and
// the descriptors name the layout, so nothing is transposed in memory.
//
// Roles (warps): one copies, one issues the matrix instructions, eight read
// the accumulators and run the epilogue; operands pass through a ring of
// stages guarded by mbarriers.  Operands that the copy engine cannot address
// (rows off 16 bytes) are first copied to aligned rows (realign.cu) where the
// caller gave a buffer: [4000, 4100] x [2044, 4100] 68 us against 221.  Without
// a buffer, and in the few calls that are estimated to be faster so, they are
// loaded by 512 more threads into the same swizzled stages, beside four
// epilogue warps, 18 bytes a cycle into an SM where the copy engine brings 50.
//
// Every wait on a barrier is bounded (tensor_core.cuh); a block whose wait ran
// out sets the call's status word, waits for what it has in flight (drain_block),
// leaves NaN in the outputs that it did not finish, and ends.
//
// Three forms:
//  vector one or two rows (decode): dot products on the CUDA cores, see
//         dot_kernel; the tensor cores' set-up would cost more than the work.
//  wide   persistent pairs of blocks over tiles of 256 x 256 (one instruction
//         spans both SMs, each holding half of either operand: a single SM
//         at 128 x 256 would need 96 bytes a cycle from L2, against the 64
//         it can take; the pair needs 64), two accumulators in tensor memory,
//         so a tile's epilogue runs under the next tile's products; or over
//         tiles of 256 x 512 on both accumulators, which needs 48 bytes a cycle.
//         8192^3 in bf16: 614 to 624 us, 1760 to 1790 TFLOP/s; bound by the clock
//         that the card's power allows.  [1024, 8192] x [8192, 8192]: 79 to 83 us, and
//         86 to 94 with bias, gelu and z, whose last stores nothing hides;
//  split  for few tiles (decode, small matrices): the output's columns take
//         the 128 accumulator lanes, its few rows the instruction's N, and a
//         cluster of up to 8 blocks splits the contraction; the partials
//         meet in distributed shared memory and are added in block order, the
//         rank-order sum of a one-shot all-reduce.  Bound by reading the
//         weights once (32 tokens of 8192 -> 8192: 24.9 us, 5.4 TB/s).
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <type_traits>

#include "activation.cuh"
#include "arx_internal.h"
#include "arx_rows.cuh"
#include "ops_launch.h"
#include "spans.h"
#include "tensor_core.cuh"

namespace arx {
namespace {

constexpr uint32_t kLanes = 128;             // rows of P in a tile (accumulator lanes)
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
  uint32_t steps;      // stages' worth of contraction: ceil(K / 64)
  uint32_t split;      // blocks of a cluster that share a tile's contraction
  uint32_t whole, pieces;  // wide form: tiles that are one piece, and pieces in all
  uint32_t tiles_p, tiles_q;
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

// ---- filling a stage by threads ---------------------------------------------------------
//
// A stage is (128 + bq) rows of eight 16-byte units; a unit's 8 elements may
// start at any even address, and end outside the matrix (zeros are filled in).
// A thread reads its units in words of 8 bytes where every row is aligned to
// them (kWord = 8), else (kWord = 2) in 4-byte words: the five around the unit,
// shifted by half a word, where it lies between words.  The addresses advance
// by a constant from stage to stage, so that a unit costs about ten
// instructions (with its address and bounds worked out anew it cost 70, which
// took the issue slots: 1.3 us a stage of 32 KB; spans.h has the arithmetic).
// Five words reach two bytes to either side of a unit.  Units of the first and
// the last stage of a contraction, which may stand at the matrix's ends, and
// units that its edge cuts (`fast` is false) take the general path, element by
// element: nothing before the matrix's first byte or past its last is read.

// A unit on its way: four words, or, where its address lies between words,
// five that are to be shifted by half a word.
struct Unit {
  uint32_t w[5];
};

// General path: element by element.
__device__ __noinline__ Unit unit_edge(const uint16_t* p, int n) {
  Unit t = {};
  const uint32_t skip = uint32_t(reinterpret_cast<uintptr_t>(p) & 2) >> 1;
  for (int i = 0; i < 8 && i < n; ++i) {
    const uint32_t v = uint32_t(p[i]) << (16 * ((i + skip) & 1));
    const uint32_t at = (i + skip) >> 1;
#pragma unroll
    for (uint32_t k = 0; k < 5; ++k)
      if (k == at) t.w[k] |= v;
  }
  return t;
}

template <int kWord>
__device__ __forceinline__ void unit_fast(Unit& t, const uint8_t* p, bool shifted) {
  if constexpr (kWord == 8) {
    const uint2 a = reinterpret_cast<const uint2*>(p)[0], b = reinterpret_cast<const uint2*>(p)[1];
    t.w[0] = a.x, t.w[1] = a.y, t.w[2] = b.x, t.w[3] = b.y;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) t.w[i] = reinterpret_cast<const uint32_t*>(p)[i];
    if (kWord == 2 && shifted) t.w[4] = reinterpret_cast<const uint32_t*>(p)[4];
  }
}

template <int kWord>
__device__ __forceinline__ void fetch(Unit& t, Place& c, const Operand& o, uint32_t stage, bool edge) {
  if (!edge && c.fast) {
    unit_fast<kWord>(t, c.at, c.shifted);
  } else {
    const uint32_t row = unit_row(o, c.id, stage * kStep), col = unit_col(o, c.id, stage * kStep);
    t = unit_edge(o.p + row * o.ld + col, unit_elements(o, row, col));
  }
  c.at += c.step;
}

template <int kWord>
__device__ __forceinline__ void put(const Unit& t, const Place& c, uint8_t* dst) {
  if (!c.on) return;
  const uint32_t line = c.id >> 3, u = c.id & 7u;
  uint4 v = make_uint4(t.w[0], t.w[1], t.w[2], t.w[3]);
  if (kWord == 2) {
    const uint32_t s = c.shifted ? 16 : 0;
    v = make_uint4(__funnelshift_r(t.w[0], t.w[1], s), __funnelshift_r(t.w[1], t.w[2], s),
                   __funnelshift_r(t.w[2], t.w[3], s), __funnelshift_r(t.w[3], t.w[4], s));
  }
  *reinterpret_cast<uint4*>(dst + line * 128 + ((u ^ (line & 7u)) << 4)) = v;  // the copy engine's swizzle
}

// ---- the roles, for one tile -------------------------------------------------------

// Bytes that the copy engine brings to a block's stage for `subs` accumulators.
__device__ __forceinline__ uint32_t copied_bytes(const GemmArgs& a, uint32_t subs) {
  return (a.p_copy ? kPBytes : 0) + (a.q_copy ? subs * a.bq * 128 : 0);
}

// One thread: the operands that the copy engine can address.  In a pair each
// block fills its own half of the stage; both halves count on the first
// block's barrier.  Returns the stages filled, fewer than last - first after a
// wait ran out.
template <bool kPair, uint32_t kSubs>
__device__ __forceinline__ uint32_t copy_tile(const GemmArgs& a, const CUtensorMap* mp, const CUtensorMap* mq, Shared& s,
                                          uint8_t* stages, Ring& ring, uint32_t p0, uint32_t q0, uint32_t first,
                                          uint32_t last, uint32_t rank) {
  const uint32_t bytes = copied_bytes(a, kSubs);
  for (uint32_t i = first; i < last; ++i) {
    if (!mbar_wait(addr_of(&s.empty[ring.slot]), ring.phase ^ 1, &s.waits)) return i - first;
    uint8_t* dst = stages + ring.slot * a.stage_bytes;
    uint32_t bar = addr_of(&s.full[ring.slot]);
    if (!kPair || rank == 0) mbar_arrive_expect(bar, kPair ? 2 * bytes : bytes);
    if (kPair) bar = cluster_peer_address(bar, 0);
    if (a.p_copy) copy_operand<kPair>(addr_of(dst), mp, a.p_layout, p0, i * kStep, kLanes, bar);
    if (a.q_copy)
#pragma unroll
      for (uint32_t j = 0; j < kSubs; ++j)
        copy_operand<kPair>(addr_of(dst) + kPBytes + j * a.bq * 128, mq, a.q_layout, q0 + j * a.bn, i * kStep, a.bq, bar);
    ring.next(a.stages);
  }
  return last - first;
}

// kLoaders threads: the operands whose rows are off 16 bytes -- both, or the
// one that the copy engine does not bring -- two units of each to a thread (bq
// <= 128).  The words of the next stages (two; one of the five-word kind) are
// in flight while a stage is stored.  Returns the stages filled, as copy_tile.
template <int kWord, bool kBoth, bool kPair>
__device__ __forceinline__ uint32_t load_tile(const GemmArgs& a, Shared& s, uint8_t* stages, Ring& ring, uint32_t p0,
                                          uint32_t q0, uint32_t first, uint32_t last, uint32_t tid) {
  constexpr int kBuffers = kWord == 2 ? 2 : 3, kUnits = kBoth ? 4 : 2;
  const bool p_first = kBoth || !a.p_copy;
  const Operand oq = operand(a.q, a.ldq, a.q_mn, a.Q, a.K, q0),
                o = p_first ? operand(a.p, a.ldp, a.p_mn, a.P, a.K, p0) : oq;
  Place c[kUnits];
#pragma unroll
  for (int j = 0; j < kUnits; ++j)
    c[j] = j < 2 ? place<kWord>(o, tid + j * kLoaders, p_first ? kLanes * 8 : a.bq * 8, first)
                 : place<kWord>(oq, tid + (j - 2) * kLoaders, a.bq * 8, first);
  Unit t[kBuffers][kUnits];
  const auto fetch_stage = [&](Unit(&u)[kUnits], uint32_t i) {
    const bool edge = i == 0 || i + 1 == a.steps;
#pragma unroll
    for (int j = 0; j < kUnits; ++j) fetch<kWord>(u[j], c[j], j < 2 ? o : oq, i, edge);
  };
#pragma unroll
  for (int b = 0; b + 1 < kBuffers; ++b)
    if (first + b < last) fetch_stage(t[b], first + b);
  for (uint32_t i = first; i < last; i += kBuffers) {
#pragma unroll
    for (int b = 0; b < kBuffers; ++b) {
      if (i + b >= last) break;
      if (i + b + kBuffers - 1 < last) fetch_stage(t[(b + kBuffers - 1) % kBuffers], i + b + kBuffers - 1);
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(addr_of(&s.empty[ring.slot]), ring.phase ^ 1, &s.waits)))
        return i + b - first;
      uint8_t* dst = stages + ring.slot * a.stage_bytes;
#pragma unroll
      for (int j = 0; j < kUnits; ++j) put<kWord>(t[b][j], c[j], j < 2 && p_first ? dst : dst + kPBytes);
      fence_async_shared();
      __syncwarp();
      const uint32_t bar = addr_of(&s.full[ring.slot]);
      if (tid % 32 == 0) {
        if (kPair)
          mbar_arrive_cluster(cluster_peer_address(bar, 0));
        else
          mbar_arrive(bar);
      }
      ring.next(a.stages);
    }
  }
  return last - first;
}

// One thread (of a pair's first block) issues the tile's products into `tmem`.
template <bool kPair, uint32_t kSubs>
__device__ __forceinline__ bool multiply_tile(const GemmArgs& a, Shared& s, uint32_t stages, Ring& ring, uint32_t tmem,
                                              uint32_t first, uint32_t last) {
  // A contraction step of 16 is 32 bytes along a K-major row, 16 rows of an
  // MN-major tile; in the descriptors' units of 16 bytes.
  const uint32_t adv_p = a.p_mn ? 128 : 2, adv_q = a.q_mn ? 128 : 2;
  for (uint32_t i = first; i < last; ++i) {
    if (!mbar_wait(addr_of(&s.full[ring.slot]), ring.phase, &s.waits)) return false;
    tmem_fence_after();
    const uint32_t base = stages + ring.slot * a.stage_bytes;
    const uint64_t dp = operand_descriptor(base, kStep * 128), dq = operand_descriptor(base + kPBytes, kStep * 128);
#pragma unroll
    for (uint32_t k = 0; k < kStep / 16; ++k) {
      mma_f16<kPair>(tmem, dp + k * adv_p, dq + k * adv_q, a.idesc, i != first || k != 0);
      if (kSubs == 2)
        mma_f16<kPair>(tmem + 256, dp + k * adv_p, dq + a.bq * 8 + k * adv_q, a.idesc, i != first || k != 0);
    }
    mma_commit<kPair>(addr_of(&s.empty[ring.slot]));
    ring.next(a.stages);
  }
  return true;
}

__device__ __forceinline__ void prefetch_l2_line(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" :: "l"(p));
}

// Loads of the residual, zero without `on`: predicated, as a load inside a
// branch is waited for where the branch ends, and volatile, so that they stay
// ahead of what they are to overlap with.
__device__ __forceinline__ uint4 load_ahead16(const void* p, bool on) {
  uint4 v;
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
      "@q ld.global.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w) : "l"(p), "r"(uint32_t(on)) : "memory");
  return v;
}
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

// The lines of a residual's row, from `col` on to `end`, on their way to L2
// while the products run, for the epilogues that read it in a chain of loops
// ([4000, 1024] x [4095, 1024]: 52.4 us without, 49.6 with).
__device__ __forceinline__ void prefetch_row(const uint16_t* row, uint32_t col, uint32_t end) {
  for (; col < end; col += 64) prefetch_l2_line(row + col);
  if (end > 0) prefetch_l2_line(row + end - 1);
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

// What 32 columns from `col` on need from memory: the bias of column col + lane
// and this lane's row of the residual.  Asked for when the last 32 columns'
// were used, so that their way overlaps with the boxes' stores, the
// accumulator's loads and the activation; asked for in place, bias and residual
// took 10 us each at [1024, 8192] x [8192, 8192] (79 us without).
struct Ahead {
  uint4 res[4];
  uint32_t bias32;
  uint16_t bias16;
};
__device__ __forceinline__ void ask(const GemmArgs& a, Ahead& h, uint32_t row, uint32_t col, bool on, uint32_t lane) {
  const bool bias = on && a.bias && col + lane < a.Q, wide = a.wdtype == ARX_F32;
  h.bias32 = load_ahead4(static_cast<const float*>(a.bias) + col + lane, bias && wide);
  h.bias16 = load_ahead2(static_cast<const uint16_t*>(a.bias) + col + lane, bias && !wide);
  const uint16_t* p = a.residual + uint64_t(row) * a.ldresidual + col;
#pragma unroll
  for (uint32_t k = 0; k < 4; ++k)
    h.res[k] = load_ahead16(p + 8 * k, on && a.residual && row < a.P && col + 8 * k < a.Q);  // Q is a multiple of 8
}

// `next`: the following 32 columns, if there are any.
template <int D>
__device__ __forceinline__ void finish_boxes(const GemmArgs& a, const CUtensorMap* mout, const CUtensorMap* mz,
                                             float (&v)[32], Ahead& ahead, uint32_t row0, uint32_t col, uint32_t next,
                                             bool more, Boxes& boxes, uint32_t lane) {
  if (a.bias) {
    const float b = a.wdtype == ARX_F32 ? __uint_as_float(ahead.bias32) : Elem<D>::widen(ahead.bias16);
#pragma unroll
    for (int k = 0; k < 32; ++k) v[k] += __shfl_sync(0xFFFFFFFFu, b, k);
  }
  if (a.z) store_box<D>(mz, v, row0, col, boxes, lane);
  activate<32>(v, a.act);
  if (a.residual) {
#pragma unroll
    for (uint32_t h = 0; h < 4; ++h) {
      const uint32_t w[4] = {ahead.res[h].x, ahead.res[h].y, ahead.res[h].z, ahead.res[h].w};
#pragma unroll
      for (uint32_t k = 0; k < 4; ++k) {
        v[8 * h + 2 * k] += Elem<D>::widen(uint16_t(w[k]));
        v[8 * h + 2 * k + 1] += Elem<D>::widen(uint16_t(w[k] >> 16));
      }
    }
  }
  ask(a, ahead, row0 + lane, next, more, lane);
  store_box<D>(mout, v, row0, col, boxes, lane);
}

// Else: a warp's 32 rows by 32 columns, staged in shared memory
// as [row][33].  A lane takes a column and walks down the rows, so that the
// warp accesses a row's line at a time; each lane on its own row, element by
// element, would touch 32 lines with every access.  kRows rows go together:
// the activation's branches and the residual's latency once for each of them
// were 230 cycles a row.
template <int D, uint32_t kRows, bool kFull>  // kFull: n >= kRows
__device__ __forceinline__ void finish_rows(const GemmArgs& a, const float* staged, uint64_t row, uint32_t n, uint32_t col,
                                            float bias) {
  uint16_t res[kRows];
  const uint16_t* p = a.residual + row * a.ldresidual + col;
  const bool on = a.residual != nullptr;
#pragma unroll
  for (uint32_t k = 0; k < kRows; ++k, p += a.ldresidual) res[k] = load_ahead2(p, on && (kFull || k < n));
  float v[kRows];
#pragma unroll
  for (uint32_t k = 0; k < kRows; ++k) v[k] = staged[k * 33] + bias;
  if (a.z) {
    uint16_t* z = a.z + row * a.ldz + col;
#pragma unroll
    for (uint32_t k = 0; k < kRows; ++k, z += a.ldz)
      if (kFull || k < n) *z = Elem<D>::round(v[k]);
  }
  activate<kRows>(v, a.act);
  if (on) {
#pragma unroll
    for (uint32_t k = 0; k < kRows; ++k) v[k] += Elem<D>::widen(res[k]);
  }
  uint16_t* out = a.out + row * a.ldout + col;
#pragma unroll
  for (uint32_t k = 0; k < kRows; ++k, out += a.ldout)
    if (kFull || k < n) *out = Elem<D>::round(v[k]);
}

template <int D, uint32_t kRows>
__device__ __forceinline__ void finish_staged(const GemmArgs& a, const float* staged, uint32_t row0, uint32_t col,
                                              uint32_t lane) {
  const uint32_t rows = row0 < a.P ? (a.P - row0 < 32 ? a.P - row0 : 32) : 0;
  if (col >= a.Q) return;
  const float bias = a.bias ? load_param(a.bias, a.wdtype, col) : 0.0f;
#pragma unroll 1
  for (uint32_t r = 0; r < rows; r += kRows) {
    if (rows - r >= kRows)
      finish_rows<D, kRows, true>(a, staged + r * 33 + lane, row0 + r, kRows, col, bias);
    else
      finish_rows<D, kRows, false>(a, staged + r * 33 + lane, row0 + r, rows - r, col, bias);
  }
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
      mbar_init(addr_of(&s.full[i]), (a.p_copy | a.q_copy) + (kTma ? 0 : (kPair ? 2 : 1) * (kLoaders / 32)));
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

constexpr uint16_t kNan16 = 0x7FFF;  // in bf16 and in fp16

// 32 rows by n columns of the outputs, by a warp.
__device__ __noinline__ void fill_nan(const GemmArgs& a, uint32_t row0, uint32_t col0, uint32_t n, uint32_t lane) {
  for (uint32_t row = row0; row < row0 + 32 && row < a.P; ++row)
    for (uint32_t c = col0 + lane; c < col0 + n && c < a.Q; c += 32) {
      a.out[row * a.ldout + c] = kNan16;
      if (a.z) a.z[row * a.ldz + c] = kNan16;
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

// Four consecutive columns of a row.  The residual's are asked for first and
// used last (res: their bits).
__device__ __forceinline__ uint2 residual4(const GemmArgs& a, uint32_t row, uint32_t col) {
  const uint16_t* p = a.residual + row * a.ldresidual + col;
  const uint32_t n = col < a.P ? a.P - col : 0;
  const bool whole = a.residual && a.quads && n >= 4, single = a.residual && !whole;
  const uint2 w = load_ahead8(p, whole);
  uint32_t r[4];
#pragma unroll
  for (uint32_t k = 0; k < 4; ++k) r[k] = load_ahead2(p + k, single && k < n);
  return make_uint2(w.x | r[0] | r[1] << 16, w.y | r[2] | r[3] << 16);
}

template <int D>
__device__ __forceinline__ void finish4(const GemmArgs& a, float (&v)[4], uint2 res, uint32_t row, uint32_t col) {
  const uint32_t n = col < a.P ? a.P - col : 0;
  const bool whole = a.quads && n >= 4;
  const auto store = [&](uint16_t* p) {
    const uint2 w = make_uint2(Elem<D>::round2(v[0], v[1]), Elem<D>::round2(v[2], v[3]));
    if (whole) {
      st_global(reinterpret_cast<uint2*>(p), w);
    } else {
      const uint32_t half[4] = {w.x & 0xFFFFu, w.x >> 16, w.y & 0xFFFFu, w.y >> 16};
#pragma unroll
      for (uint32_t k = 0; k < 4; ++k)
        if (k < n) p[k] = uint16_t(half[k]);
    }
  };
#pragma unroll
  for (uint32_t k = 0; k < 4; ++k)
    if (a.bias && k < n) v[k] += load_param(a.bias, a.wdtype, col + k);
  if (a.z) store(a.z + row * a.ldz + col);
  activate<4>(v, a.act);
  if (a.residual) {
    v[0] += Elem<D>::widen(uint16_t(res.x)), v[1] += Elem<D>::widen(uint16_t(res.x >> 16));
    v[2] += Elem<D>::widen(uint16_t(res.y)), v[3] += Elem<D>::widen(uint16_t(res.y >> 16));
  }
  store(a.out + row * a.ldout + col);
}

// kSubs: accumulators to a tile.
template <int D, int kWord, bool kBoth, uint32_t kSubs>
__global__ void __launch_bounds__(kGemmThreads<kWord == 16>, 1)
    gemm_wide_kernel(const __grid_constant__ GemmArgs a, const __grid_constant__ CUtensorMap mp,
                     const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mout,
                     const __grid_constant__ CUtensorMap mz) {
  constexpr bool kTma = kWord == 16;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared s;
  uint8_t* stages = smem_raw + ((1024u - (addr_of(smem_raw) & 1023u)) & 1023u);
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x & 31, rank = cluster_ctarank();
  setup<kTma, true>(a, &mp, &mq, s, warp);
  dependent_launch_prologue();
  const uint32_t pieces = a.pieces, first_piece = blockIdx.x / 2, step = gridDim.x / 2;

  Ring ring;
  const bool copies = threadIdx.x == 0 && (a.p_copy | a.q_copy), loads = !kTma && threadIdx.x >= kFirstLoader<kTma>;
  if (copies || loads) {
    uint32_t t = first_piece, filled = 0;
    for (; t < pieces; t += step) {
      const Piece w = piece_at<kSubs>(a, t);
      const uint32_t p0 = (2 * w.tp + rank) * kLanes, q0 = w.q0 + rank * a.bq;
      filled = 0;
      if (copies && kSubs == 2 && w.subs == 2)
        filled = copy_tile<true, kSubs>(a, &mp, &mq, s, stages, ring, p0, q0, 0, a.steps, rank);
      else if (copies)
        filled = copy_tile<true, 1>(a, &mp, &mq, s, stages, ring, p0, q0, 0, a.steps, rank);
      else if constexpr (!kTma)
        filled = load_tile<kWord, kBoth, true>(a, s, stages, ring, p0, q0, 0, a.steps, threadIdx.x - kFirstLoader<kTma>);
      if (filled < a.steps) break;
    }
    note_fills<kTma>(s, (t - first_piece) / step * a.steps + (t < pieces ? filled : 0), copies, warp, lane);
  } else if (warp == 1 && lane == 0 && rank == 0 && a.steps > 0) {
    uint32_t n = 0;
    for (uint32_t t = first_piece; t < pieces; t += step, ++n) {
      // One accumulator to a tile: two tiles' alternate.  Two: the tile has both.
      const uint32_t b = kSubs == 2 ? 0 : n & 1, use = kSubs == 2 ? n : n >> 1;
      if (!mbar_wait(addr_of(&s.acc_empty[b]), (use & 1) ^ 1, &s.waits)) break;
      tmem_fence_after();
      const uint32_t subs = piece_at<kSubs>(a, t).subs;
      if (!(kSubs == 2 && subs == 2 ? multiply_tile<true, kSubs>(a, s, addr_of(stages), ring, s.tmem, 0, a.steps)
                                    : multiply_tile<true, 1>(a, s, addr_of(stages), ring, s.tmem + b * 256, 0, a.steps)))
        break;
      mma_commit<true>(addr_of(&s.acc_full[b]));
    }
  } else if (warp >= 2 && warp < 2 + kEpilogueWarps<kTma>) {
    const uint32_t quarter = warp & 3;  // the accumulator lanes this warp may read
    float* staged = reinterpret_cast<float*>(stages + a.stages * a.stage_bytes) + (warp - 2) * 32 * 33;
    Boxes boxes{addr_of(stages + a.stages * a.stage_bytes) + (warp - 2) * 4096, 0};
    uint32_t n = 0, t = first_piece;
    for (; t < pieces; t += step, ++n) {
      const Piece w = piece_at<kSubs>(a, t);
      const uint32_t b = kSubs == 2 ? 0 : n & 1, use = kSubs == 2 ? n : n >> 1;
      const uint32_t row0 = (2 * w.tp + rank) * kLanes + quarter * 32;
      const uint32_t half = kTma ? a.bn / 2 : a.bn, c0 = kTma ? (warp - 2) / 4 * half : 0;
      // The warp's runs of 32 columns: `half` of each accumulator.
      const uint32_t runs = row0 < a.P ? w.subs * (half / 32) : 0;
      const auto column = [&](uint32_t i) {
        const uint32_t j = i * 32 >= half;
        return w.q0 + j * a.bn + c0 + i * 32 - j * half;
      };
      if (!(kTma && a.octets) && a.residual && row0 + lane < a.P && warp < 6) {
        const uint32_t end = w.q0 + w.subs * a.bn;
        prefetch_row(a.residual + (row0 + lane) * a.ldresidual, w.q0, end < a.Q ? end : a.Q);
      }
      Ahead ahead;
      if (kTma && a.octets) ask(a, ahead, row0 + lane, column(0), runs > 0, lane);
      if (a.steps > 0) {
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(addr_of(&s.acc_full[b]), use & 1, &s.waits))) break;
        tmem_fence_after();
      }
      for (uint32_t i = 0; i < runs; ++i) {
        const uint32_t col = column(i), acc = s.tmem + b * 256 + (quarter * 32 << 16) + (col - w.q0);
        if (col >= a.Q) break;  // and so are those after it
        if (kTma && a.octets) {
          float v[32];
          if (a.steps > 0) {
            uint32_t lo[16], hi[16];
            tmem_load16_start(acc, lo);
            tmem_load16_start(acc + 16, hi);
            tmem_load_wait(lo);
            tmem_load_wait(hi);
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(lo[k]), v[16 + k] = __uint_as_float(hi[k]);
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = 0.0f;
          }
          finish_boxes<D>(a, &mout, &mz, v, ahead, row0, col, column(i + 1), i + 1 < runs, boxes, lane);
        } else {
          __syncwarp();
#pragma unroll
          for (uint32_t h = 0; h < 32; h += 16) {
            float v[16] = {};
            if (a.steps > 0) tmem_load16(acc + h, v);
#pragma unroll
            for (int k = 0; k < 16; ++k) staged[lane * 33 + h + k] = v[k];
          }
          __syncwarp();
          finish_staged<D, kTma ? 16 : 8>(a, staged, row0, col + lane, lane);
        }
      }
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(cluster_peer_address(addr_of(&s.acc_empty[b]), 0));
    }
    for (; t < pieces; t += step) {  // after a wait ran out
      const Piece w = piece_at<kSubs>(a, t);
      const uint32_t half = kTma ? a.bn / 2 : a.bn, c0 = kTma ? (warp - 2) / 4 * half : 0;
      for (uint32_t j = 0; j < w.subs; ++j)
        fill_nan(a, (2 * w.tp + rank) * kLanes + quarter * 32, w.q0 + j * a.bn + c0, half, lane);
    }
    if (kTma && lane == 0) bulk_wait_all();
  }
  __syncwarp();
  finish_block<kTma, true, kSubs>(a, s, warp, rank);
}

// One tile per cluster; block r of the cluster takes the r-th share of the
// contraction.  P's rows are the output's columns here, Q's rows its rows.
template <int D, int kWord, bool kBoth>
__global__ void __launch_bounds__(kGemmThreads<kWord == 16>, kWord == 16 ? 2 : 1)
    gemm_split_kernel(const __grid_constant__ GemmArgs a, const __grid_constant__ CUtensorMap mp,
                      const __grid_constant__ CUtensorMap mq) {
  constexpr bool kTma = kWord == 16;
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
  const bool copies = threadIdx.x == 0 && (a.p_copy | a.q_copy), loads = !kTma && threadIdx.x >= kFirstLoader<kTma>;
  if (copies) {
    note_fills<kTma>(s, copy_tile<false, 1>(a, &mp, &mq, s, stages, ring, p0, q0, first, last, 0), true, warp, lane);
  } else if (loads) {
    if constexpr (!kTma) {
      const uint32_t tid = threadIdx.x - kFirstLoader<kTma>;
      note_fills<kTma>(s, load_tile<kWord, kBoth, false>(a, s, stages, ring, p0, q0, first, last, tid), false, warp, lane);
    }
  } else if (warp == 1 && lane == 0 && first < last) {
    if (multiply_tile<false, 1>(a, s, addr_of(stages), ring, s.tmem, first, last))
      mma_commit<false>(addr_of(&s.acc_full[0]));
  } else if (warp >= 2 && warp < 2 + kEpilogueWarps<kTma>) {
    const uint32_t quarter = warp & 3;
    if (a.residual)
      for (uint32_t i = rank * 32 * kEpilogueWarps<kTma> + threadIdx.x - 64; i < a.bn && q0 + i < a.Q;
           i += a.split * 32 * kEpilogueWarps<kTma>)
        prefetch_row(a.residual + (q0 + i) * a.ldresidual, p0, p0 + kLanes < a.P ? p0 + kLanes : a.P);
    bool ok = true;
    if (first < last) {
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(addr_of(&s.acc_full[0]), 0, &s.waits));
      tmem_fence_after();
    }
    if (ok)
      for (uint32_t c = (warp - 2) / 4 * 16; c < a.bn; c += kEpilogueWarps<kTma> * 4) {
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
  if (s.waits.abort) {  // its part of every sum is NaN, once nothing lands on it any more
    drain_block<kTma, false, 1>(a, s);
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < a.bn * kLanes; i += kGemmThreads<kTma>) part[i] = __int_as_float(0x7FFFFFFF);
    __syncthreads();
  }
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
    const uint2 res = residual4(a, row, j);
    float4 in[8];
#pragma unroll
    for (uint32_t r = 0; r < 8; ++r)
      if (r < a.split) in[r] = ld_cluster_f32x4(cluster_peer_address(at + i * 16, r));
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (uint32_t r = 0; r < 8; ++r)
      if (r < a.split) v[0] += in[r].x, v[1] += in[r].y, v[2] += in[r].z, v[3] += in[r].w;
    finish4<D>(a, v, res, row, j);
  }
  finish_block<kTma, false, 1>(a, s, warp, rank);
}

// ---- one or two rows --------------------------------------------------------------------
//
// out[m][j] = sum_k x[m][k] w[j][k]: w is read once, which bounds the kernel,
// at 2 M operations to an element.  Two tokens of 4096 -> 2048: 4.6 us, the
// split form 5.8; three: 5.3, but 33 against 25 at 8192 x 8192.  A warp (or `split` warps of a block) takes
// a feature j; its lanes take 16-byte units of the row, kBatch of them in
// flight, and x comes from L1.  The lanes' sums meet in a butterfly and the
// split warps' in warp order.  kV = 1: rows off 16 bytes, element by element.

constexpr uint32_t kDotRows = 2;
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
  // The lanes' first batch of the row: asked for whole, rows of 16 KB came
  // twice (one token, 8192 x 8192: 34.6 us against 23.5; none 26.0).
  if (kV == 8 && share == 0 && lane == 0 && j < a.Q && a.K > 0)
    prefetch_l2_bulk(a.q + j * a.ldq, a.K < 2048 ? a.K * 2 : 4096);
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

// Map of an operand of `rows` by `k`, for tiles of `tile` rows by 64 of the
// contraction.
cudaError_t encode(CUtensorMap* m, uint32_t* layout, const uint16_t* base, uint64_t ld, uint32_t rows, uint32_t k,
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

// Map of an output, for boxes of 32 rows by 32 columns.
cudaError_t encode_output(CUtensorMap* m, uint16_t* base, uint64_t ld, uint32_t rows, uint32_t cols, bool bf16) {
  cudaError_t err = cudaSuccess;
  auto f = encode_function(&err);
  if (!f) return err;
  const cuuint64_t dims[2] = {cols, rows}, strides[1] = {(rows > 1 ? ld : cols) * 2};
  const cuuint32_t box[2] = {32, 32}, el[2] = {1, 1};
  const CUresult r = f(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, base, dims,
                       strides, box, el, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
                       CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

bool copyable(const uint16_t* p, uint64_t ld, uint64_t nrows) {
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

// A persistent grid: as many pairs as the device holds at once (two blocks to
// a pair, one block to an SM), or fewer tiles.
template <int D, int kWord, bool kBoth, uint32_t kSubs>
cudaError_t launch_wide(const GemmArgs& a, const CUtensorMap (&m)[4], int sms, cudaStream_t st) {
  const uint32_t tiles = a.tiles_p * a.tiles_q, pairs = uint32_t(sms) / 2, rest = tiles % pairs;
  const bool halves = kSubs == 2 && 2 * rest <= pairs;
  GemmArgs g = a;
  g.whole = halves ? tiles - rest : tiles;
  g.pieces = halves ? tiles + rest : tiles;
  uint32_t smem = 1024 + g.stages * g.stage_bytes + kEpilogueWarps<kWord == 16> * kStagedBytes;
  if (smem < kAloneShared) smem = kAloneShared;
  return launch_cluster<gemm_wide_kernel<D, kWord, kBoth, kSubs>>(2 * (g.pieces < pairs ? g.pieces : pairs),
                                                                 kGemmThreads<kWord == 16>, 2, smem, st, g, m[0], m[1],
                                                                 m[2], m[3]);
}

template <int D, int kWord, bool kBoth>
cudaError_t launch_split(const GemmArgs& a, const CUtensorMap (&m)[4], cudaStream_t st) {
  return launch_cluster<gemm_split_kernel<D, kWord, kBoth>>(a.tiles_p * a.tiles_q * a.split,
                                                            kGemmThreads<kWord == 16>, a.split,
                                                            1024 + a.stages * a.stage_bytes, st, a, m[0], m[1]);
}

uint32_t ceil_div(uint64_t a, uint64_t b) { return uint32_t((a + b - 1) / b); }

// Which form, with how many rows of Q to a tile and how many blocks to a
// tile's contraction: the one with the least estimated time, in SM cycles, on
// 152 SMs (a constant: the form decides the order of a sum).
struct Form {
  bool wide;
  uint32_t bn, split, subs;
  double cycles;
};

Form choose_form(const GemmCall& c, uint32_t steps, bool p_copy, bool q_copy) {
  constexpr uint32_t sms = 152;
  Form best{};
  const auto consider = [&](const Form& f) {
    if (best.bn == 0 || f.cycles < best.cycles) best = f;
  };
  // A stage of `rows` rows of c.p and `cols` of c.q costs its copies or its
  // products (2.1 cycles a row of the kernel's Q), whichever is longer.
  // Measured, bytes a cycle into an SM: 46 in pairs when all of them are at
  // work, 53 for half of them, a seventh less with 128 rows of Q; 41 for a
  // split block alone on its SM, 55 for one with the whole shared memory, 66 for
  // two; through loading threads 16 (12 in pairs, where the slower of two blocks
  // counts).
  const bool threads = !p_copy || !q_copy;
  const auto stage = [&](uint32_t rows, uint32_t cols, uint32_t bn, double engine, double loaded) {
    const double copies = rows * 128.0 / (p_copy ? engine : loaded) + cols * 128.0 / (q_copy ? engine : loaded);
    return copies > 2.1 * bn ? copies : 2.1 * bn;
  };
  // Starting and ending a block takes about 6000 cycles, joining and storing a
  // tile 25 a row of Q, 30 to 40 through a cluster; of a wide tile all but the last
  // run under the next one's products, 2800 + 7 a row at the least.
  constexpr uint32_t pairs = sms / 2;
  for (uint32_t bn = 256; bn >= 128; bn /= 2) {
    const uint32_t tiles = ceil_div(c.rows, 2 * kLanes) * ceil_div(c.cols, bn);
    const double engine = (58 - 12.0 * (tiles < pairs ? tiles : pairs) / pairs) * (bn == 128 ? 0.86 : 1);
    const double products = steps * stage(kLanes, bn / 2, bn, engine, 12), store = 2800 + 7 * bn;
    consider({true, bn, 1, 1, ceil_div(tiles, pairs) * (products > store ? products : store) + 6000 + 25 * bn});
  }
  // Two accumulators to a tile: 1290 cycles a stage (630 us against 681 at
  // 8192^3, where the card's power sets the clock), and no tile's epilogue runs
  // under the next one's products.
  if (!threads) {
    const uint32_t tiles = ceil_div(c.rows, 2 * kLanes) * ceil_div(c.cols, 512), rest = tiles % pairs;
    const bool halves = rest && 2 * rest <= pairs;
    const double rounds = tiles / pairs + (rest && !halves);
    consider({true, 256, 1, 2,
              rounds * (steps * 1290.0 + 4000) + (halves ? steps * 712.0 + 4000 : 0) + 6000 + 25 * 256});
  }
  for (uint32_t bn = c.p_mn ? 64 : 16; bn <= (threads ? 128 : 256); bn *= 2) {
    const uint32_t tiles = ceil_div(c.cols, kLanes) * ceil_div(c.rows, bn);
    const bool two = !threads && bn <= 128;  // blocks to an SM
    for (uint32_t split = 1; split <= 8 && (split == 1 || split <= steps); split *= 2) {
      // Clusters at work at once: those of 4 and 8 leave some SMs of a processing
      // cluster over.
      const uint32_t at_once = two ? (split == 8 ? 36 : split == 4 ? 72 : 2 * sms / split)
                                   : (split == 8 ? 14 : split == 4 ? 36 : sms / split);
      const double join = (split == 8 ? 40 : split > 1 ? 30 : 25) * bn;
      const uint32_t rounds = ceil_div(tiles, at_once);
      const double on_sm = !two ? rounds : rounds > 1 ? 2 * rounds : ceil_div(uint64_t(tiles) * split, sms);
      const double engine = two && on_sm > 1 ? 66 : bn > 128 ? 55 : 41;
      const double own = ceil_div(steps, split) * stage(bn, kLanes, bn, engine, 16) + join;
      consider({false, bn, split, 1, two ? on_sm * own + 6000 : on_sm * (own + 6000)});
    }
    if (bn >= c.rows) break;
  }
  return best;
}

// Does the dot form take the call, and with units of 8 elements?
bool dot_units(const GemmCall& c) {
  return c.k % 8 == 0 && copyable(static_cast<const uint16_t*>(c.p), c.ldp, c.rows) &&
         copyable(static_cast<const uint16_t*>(c.q), c.ldq, c.cols);
}
bool dot_form(const GemmCall& c) {
  // Element by element the dot form is the slower one from about 8 million
  // weights (one token of 4099 -> 2047: 15.9 us against the split form's 15.6;
  // of 8193 -> 8191: 138 against 49).
  return c.rows <= kDotRows && !c.p_mn && !c.q_mn && (dot_units(c) || c.cols * c.k < (uint64_t(1) << 23));
}

// The copy engine takes operands whose rows are on 16 bytes; an empty one has no map.
bool p_copyable(const GemmCall& c) {
  return c.k > 0 && copyable(static_cast<const uint16_t*>(c.p), c.ldp, c.p_mn ? c.k : c.rows);
}
bool q_copyable(const GemmCall& c) {
  return c.k > 0 && copyable(static_cast<const uint16_t*>(c.q), c.ldq, c.q_mn ? c.k : c.cols);
}

// Operands to be brought onto rows of 16 bytes first: the set with the least
// estimated time of copies and product.  Copies count as 2.3 us and 2.9 TB/s
// (17.9 MB measured 6 us).
// Forms with loading threads are estimated for long contractions from L2; short
// ones and cold weights take half as long again, and their first words 3 us
// ([4, 515] x [1000, 515]: 13 us against 4.5 on aligned rows).
struct Copies {
  bool p, q;
  uint64_t p_bytes, q_bytes;  // 0 for an operand that stays
};
uint64_t copy_pitch(uint64_t inner) { return (inner + 7) / 8 * 8; }

Copies choose_copies(const GemmCall& c) {
  const bool p_copy = p_copyable(c), q_copy = q_copyable(c);
  Copies best{};
  if (c.rows == 0 || c.cols == 0 || c.k == 0 || (p_copy && q_copy) || dot_form(c)) return best;
  const uint32_t steps = ceil_div(c.k, kStep);
  const uint64_t p_bytes = (c.p_mn ? c.k * copy_pitch(c.rows) : c.rows * copy_pitch(c.k)) * 2,
                 q_bytes = (c.q_mn ? c.k * copy_pitch(c.cols) : c.cols * copy_pitch(c.k)) * 2;
  const auto estimate = [&](bool p, bool q) {
    const double cycles = choose_form(c, steps, p, q).cycles;
    return p && q ? cycles : 1.5 * cycles + 6000;
  };
  double least = estimate(p_copy, q_copy);
  for (int set = 1; set < 4; ++set) {
    const bool p = set & 1, q = set & 2;
    if ((p && p_copy) || (q && q_copy)) continue;
    const uint64_t bytes = (p ? p_bytes : 0) + (q ? q_bytes : 0);
    const double cycles = estimate(p_copy || p, q_copy || q) + 4400 + double(bytes) / 1550;
    if (cycles < least) least = cycles, best = {p, q, p ? p_bytes : 0, q ? q_bytes : 0};
  }
  return best;
}

template <int D, int kV>
cudaError_t launch_dot(const GemmArgs& a, cudaStream_t st) {
  const dim3 grid(ceil_div(a.Q, kDotThreads / 32 / a.split));
  return a.P == 1 ? launch_op(dot_kernel<D, 1, kV>, grid, kDotThreads, 0, st, a)
                  : launch_op(dot_kernel<D, 2, kV>, grid, kDotThreads, 0, st, a);
}

}  // namespace

size_t gemm_copies_bytes(const GemmCall& c) {
  const Copies k = choose_copies(c);
  return size_t((k.p_bytes + 15) / 16 * 16 + k.q_bytes);
}

cudaError_t launch_gemm(const GemmCall& c, cudaStream_t st) {
  cudaError_t err = cudaSuccess;
  if (c.copies) {
    const Copies k = choose_copies(c);
    if (k.p || k.q) {
      GemmCall on = c;
      on.copies = nullptr;
      RealignPair r{};
      const auto add = [&](const void* src, uint64_t ld, uint64_t rows, uint64_t cols, void* dst) {
        r.m[r.n++] = {static_cast<const uint16_t*>(src), static_cast<uint16_t*>(dst), rows, ld, copy_pitch(cols),
                      int64_t(cols)};
      };
      if (k.p) {
        add(c.p, c.ldp, c.p_mn ? c.k : c.rows, c.p_mn ? c.rows : c.k, c.copies);
        on.p = c.copies, on.ldp = r.m[0].ld_dst;
      }
      if (k.q) {
        void* dst = static_cast<uint8_t*>(c.copies) + (k.p_bytes + 15) / 16 * 16;
        add(c.q, c.ldq, c.q_mn ? c.k : c.cols, c.q_mn ? c.cols : c.k, dst);
        on.q = dst, on.ldq = r.m[r.n - 1].ld_dst;
      }
      err = launch_realign(r, st);
      return err != cudaSuccess ? err : launch_gemm(on, st);
    }
  }
  const int sms = current_sm_count(&err);
  if (sms < 1) return err;
  GemmArgs a{};
  a.out = static_cast<uint16_t*>(c.out);
  a.z = static_cast<uint16_t*>(c.z);
  a.bias = c.bias;
  a.residual = static_cast<const uint16_t*>(c.residual);
  a.ldout = c.ldout, a.ldz = c.ldz, a.ldresidual = c.ldresidual;
  a.status = c.status;
  a.wait_ns = c.wait_ns;
  a.act = c.act, a.wdtype = c.wdtype;
  a.K = uint32_t(c.k);
  a.steps = ceil_div(c.k, kStep);

  const auto aligned = [](const void* p, uint64_t ld, unsigned elements) {
    return !p || (reinterpret_cast<uintptr_t>(p) % (2 * elements) == 0 && ld % elements == 0);
  };
  const auto out_aligned = [&](unsigned n) {
    return aligned(a.out, a.ldout, n) && aligned(a.z, a.ldz, n) && aligned(a.residual, a.ldresidual, n);
  };
  a.quads = out_aligned(4);
  a.octets = out_aligned(8) && c.cols % 8 == 0 && reinterpret_cast<uintptr_t>(a.bias) % 16 == 0;

  const bool bf16 = c.dtype == ARX_BF16;
  if (dot_form(c)) {
    const bool units = dot_units(c);
    a.p = static_cast<const uint16_t*>(c.p), a.q = static_cast<const uint16_t*>(c.q);
    a.ldp = c.ldp, a.ldq = c.ldq;
    a.P = uint32_t(c.rows), a.Q = uint32_t(c.cols);
    // Warps for about 16 to an SM, while each keeps 256 elements or more.
    a.split = 1;
    while (a.split < 8 && uint64_t(a.Q) * a.split < 2432 && a.K / a.split > 512) a.split *= 2;
    if (bf16) return units ? launch_dot<ARX_BF16, 8>(a, st) : launch_dot<ARX_BF16, 1>(a, st);
    return units ? launch_dot<ARX_F16, 8>(a, st) : launch_dot<ARX_F16, 1>(a, st);
  }

  const auto *cp = static_cast<const uint16_t*>(c.p), *cq = static_cast<const uint16_t*>(c.q);
  // Threads read what the copy engine cannot, in words of 8 bytes where every
  // row is aligned to them.
  const uint64_t cp_rows = c.p_mn ? a.K : c.rows, cq_rows = c.q_mn ? a.K : c.cols;
  const bool cp_copy = p_copyable(c), cq_copy = q_copyable(c);
  uint64_t bits = 0;
  if (!cp_copy) bits |= reinterpret_cast<uintptr_t>(cp) | (cp_rows > 1 ? c.ldp * 2 : 0);
  if (!cq_copy) bits |= reinterpret_cast<uintptr_t>(cq) | (cq_rows > 1 ? c.ldq * 2 : 0);
  const uint32_t word = cp_copy && cq_copy ? 16 : bits % 8 == 0 ? 8 : 2;
  const Form form = choose_form(c, a.steps, cp_copy, cq_copy);
  const bool wide = form.wide;
  a.bn = form.bn;
  a.split = form.split;
  if (wide) {
    a.p = cp, a.q = cq, a.ldp = c.ldp, a.ldq = c.ldq, a.p_mn = c.p_mn, a.q_mn = c.q_mn;
    a.P = uint32_t(c.rows), a.Q = uint32_t(c.cols);
    a.p_copy = cp_copy, a.q_copy = cq_copy;
    a.bq = a.bn / 2;
    a.tmem_columns = 512;
  } else {
    a.p = cq, a.q = cp, a.ldp = c.ldq, a.ldq = c.ldp, a.p_mn = c.q_mn, a.q_mn = c.p_mn;
    a.P = uint32_t(c.cols), a.Q = uint32_t(c.rows);
    a.p_copy = cq_copy, a.q_copy = cp_copy;
    a.bq = a.bn;
    a.tmem_columns = a.bn < 32 ? 32 : a.bn;
  }
  const uint32_t lanes = wide ? 2 * kLanes : kLanes;
  a.tiles_p = ceil_div(a.P, lanes);
  a.tiles_q = ceil_div(a.Q, form.subs * a.bn);
  a.stage_bytes = kPBytes + form.subs * a.bq * 128;
  a.stages = (word != 16 ? kLoadedBudget : wide || a.bn > 128 ? kStageBudget : kSplitBudget) / a.stage_bytes;
  if (a.stages > kMaxStages) a.stages = kMaxStages;
  a.idesc = mma_descriptor(c.dtype == ARX_BF16, a.p_mn, a.q_mn, lanes, a.bn);

  CUtensorMap m[4] = {};  // P, Q, out, z
  if (a.p_copy) {
    err = encode(&m[0], &a.p_layout, a.p, a.ldp, a.P, a.K, a.p_mn, kLanes, bf16);
    if (err != cudaSuccess) return err;
  }
  if (a.q_copy) {
    err = encode(&m[1], &a.q_layout, a.q, a.ldq, a.Q, a.K, a.q_mn, a.bq, bf16);
    if (err != cudaSuccess) return err;
  }
  if (wide && word == 16 && a.octets) {
    err = encode_output(&m[2], a.out, a.ldout, a.P, a.Q, bf16);
    if (err == cudaSuccess && a.z) err = encode_output(&m[3], a.z, a.ldz, a.P, a.Q, bf16);
    if (err != cudaSuccess) return err;
  }
  const auto run = [&](auto w, auto both) {
    constexpr int kWord = decltype(w)::value;
    constexpr bool kBoth = decltype(both)::value;
    if constexpr (kWord == 16)
      if (wide && form.subs == 2)
        return bf16 ? launch_wide<ARX_BF16, kWord, kBoth, 2>(a, m, sms, st)
                    : launch_wide<ARX_F16, kWord, kBoth, 2>(a, m, sms, st);
    if (wide)
      return bf16 ? launch_wide<ARX_BF16, kWord, kBoth, 1>(a, m, sms, st)
                  : launch_wide<ARX_F16, kWord, kBoth, 1>(a, m, sms, st);
    return bf16 ? launch_split<ARX_BF16, kWord, kBoth>(a, m, st) : launch_split<ARX_F16, kWord, kBoth>(a, m, st);
  };
  using std::integral_constant;
  const bool both = !cp_copy && !cq_copy;
  if (word == 16) return run(integral_constant<int, 16>{}, integral_constant<bool, false>{});
  if (word == 8)
    return both ? run(integral_constant<int, 8>{}, integral_constant<bool, true>{})
                : run(integral_constant<int, 8>{}, integral_constant<bool, false>{});
  return both ? run(integral_constant<int, 2>{}, integral_constant<bool, true>{})
              : run(integral_constant<int, 2>{}, integral_constant<bool, false>{});
}

}  // namespace arx
