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
// The parts that the gated block's products (gated.cu) share are in gemm.cuh; its
// backward pass also takes two products in one launch of these kernels (Extra).
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

#include <type_traits>

#include "activation.cuh"
#include "gemm.cuh"

namespace arx {
namespace {

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

// The lines of a residual's row, from `col` on to `end`, on their way to L2
// while the products run, for the epilogues that read it in a chain of loops
// ([4000, 1024] x [4095, 1024]: 52.4 us without, 49.6 with).
__device__ __forceinline__ void prefetch_row(const uint16_t* row, uint32_t col, uint32_t end) {
  for (; col < end; col += 64) prefetch_l2_line(row + col);
  if (end > 0) prefetch_l2_line(row + end - 1);
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
__device__ __forceinline__ void finish_rows(const GemmArgs& a, const Output& o, const float* staged, uint64_t row, uint32_t n, uint32_t col,
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
  uint16_t* out = o.p + row * o.ld + col;
#pragma unroll
  for (uint32_t k = 0; k < kRows; ++k, out += o.ld)
    if (kFull || k < n) *out = Elem<D>::round(v[k]);
}

template <int D, uint32_t kRows>
__device__ __forceinline__ void finish_staged(const GemmArgs& a, const Output& o, const float* staged, uint32_t row0, uint32_t col,
                                              uint32_t lane) {
  const uint32_t rows = row0 < a.P ? (a.P - row0 < 32 ? a.P - row0 : 32) : 0;
  if (col >= a.Q) return;
  const float bias = a.bias ? load_param(a.bias, a.wdtype, col) : 0.0f;
#pragma unroll 1
  for (uint32_t r = 0; r < rows; r += kRows) {
    if (rows - r >= kRows)
      finish_rows<D, kRows, true>(a, o, staged + r * 33 + lane, row0 + r, kRows, col, bias);
    else
      finish_rows<D, kRows, false>(a, o, staged + r * 33 + lane, row0 + r, rows - r, col, bias);
  }
}

constexpr uint16_t kNan16 = 0x7FFF;  // in bf16 and in fp16

// 32 rows by n columns of the outputs, by a warp.
__device__ __noinline__ void fill_nan(const GemmArgs& a, Output o, uint32_t row0, uint32_t col0, uint32_t n,
                                      uint32_t lane) {
  for (uint32_t row = row0; row < row0 + 32 && row < a.P; ++row)
    for (uint32_t c = col0 + lane; c < col0 + n && c < a.Q; c += 32) {
      o.p[row * o.ld + c] = kNan16;
      if (a.z) a.z[row * a.ldz + c] = kNan16;
    }
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
__device__ __forceinline__ void finish4(const GemmArgs& a, const Output& o, float (&v)[4], uint2 res, uint32_t row, uint32_t col) {
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
  store(o.p + row * o.ld + col);
}

// kSubs: accumulators to a tile.
template <int D, int kWord, bool kBoth, uint32_t kSubs, int kExtra>
__global__ void __launch_bounds__(kGemmThreads<kWord == 16>, 1)
    gemm_wide_kernel(const __grid_constant__ GemmArgs a, const __grid_constant__ CUtensorMap mp,
                     const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mout,
                     const __grid_constant__ CUtensorMap mz, const __grid_constant__ SecondMaps<kExtra> m2) {
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
      Piece w = piece_at<kSubs>(a, t);
      const CUtensorMap* p = &mp;
      if constexpr (kExtra == kStack)
        if (second_product<kExtra>(a, w.tp)) p = &m2.in;
      const uint32_t p0 = (2 * w.tp + rank) * kLanes, q0 = w.q0 + rank * a.bq;
      filled = 0;
      if (copies && kSubs == 2 && w.subs == 2)
        filled = copy_tile<true, kSubs, kExtra>(a, p, &mq, &m2, s, stages, ring, p0, q0, 0, a.steps, rank);
      else if (copies)
        filled = copy_tile<true, 1, kExtra>(a, p, &mq, &m2, s, stages, ring, p0, q0, 0, a.steps, rank);
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
      Piece w = piece_at<kSubs>(a, t);
      const bool second = second_product<kExtra>(a, w.tp);
      const Output o = output_of<kExtra>(a, second);
      const CUtensorMap* map = &mout;
      if constexpr (kExtra == kStack)
        if (second) map = &m2.out;
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
          finish_boxes<D>(a, map, &mz, v, ahead, row0, col, column(i + 1), i + 1 < runs, boxes, lane);
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
          finish_staged<D, kTma ? 16 : 8>(a, o, staged, row0, col + lane, lane);
        }
      }
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(cluster_peer_address(addr_of(&s.acc_empty[b]), 0));
    }
    for (; t < pieces; t += step) {  // after a wait ran out
      Piece w = piece_at<kSubs>(a, t);
      const Output o = output_of<kExtra>(a, second_product<kExtra>(a, w.tp));
      const uint32_t half = kTma ? a.bn / 2 : a.bn, c0 = kTma ? (warp - 2) / 4 * half : 0;
      for (uint32_t j = 0; j < w.subs; ++j)
        fill_nan(a, o, (2 * w.tp + rank) * kLanes + quarter * 32, w.q0 + j * a.bn + c0, half, lane);
    }
    if (kTma && lane == 0) bulk_wait_all();
  }
  __syncwarp();
  finish_block<kTma, true, kSubs>(a, s, warp, rank);
}

// One tile per cluster; block r of the cluster takes the r-th share of the
// contraction.  P's rows are the output's columns here, Q's rows its rows.
template <int D, int kWord, bool kBoth, int kExtra>
__global__ void __launch_bounds__(kGemmThreads<kWord == 16>, kWord == 16 ? 2 : 1)
    gemm_split_kernel(const __grid_constant__ GemmArgs a, const __grid_constant__ CUtensorMap mp,
                      const __grid_constant__ CUtensorMap mq, const __grid_constant__ SecondMaps<kExtra> m2) {
  constexpr bool kTma = kWord == 16;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared s;
  uint8_t* stages = smem_raw + ((1024u - (addr_of(smem_raw) & 1023u)) & 1023u);
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  setup<kTma, false>(a, &mp, &mq, s, warp);
  dependent_launch_prologue();
  const uint32_t rank = blockIdx.x % a.split, tile = blockIdx.x / a.split;
  const uint32_t tp = tile % a.tiles_p;
  uint32_t tq = tile / a.tiles_p;
  const bool second = second_product<kExtra>(a, tq);
  const Output o = output_of<kExtra>(a, second);
  const uint32_t p0 = tp * kLanes, q0 = tq * a.bn;
  const uint32_t share = (a.steps + a.split - 1) / a.split;
  const uint32_t first = rank * share < a.steps ? rank * share : a.steps;
  const uint32_t last = first + share < a.steps ? first + share : a.steps;
  float* part = reinterpret_cast<float*>(stages);  // [bn][128 lanes], once the stages are done with

  Ring ring;
  const bool copies = threadIdx.x == 0 && (a.p_copy | a.q_copy), loads = !kTma && threadIdx.x >= kFirstLoader<kTma>;
  if (copies) {
    const CUtensorMap* q = &mq;
    if constexpr (kExtra == kStack)
      if (second) q = &m2.in;
    const uint32_t filled = copy_tile<false, 1, kExtra>(a, &mp, q, &m2, s, stages, ring, p0, q0, first, last, 0);
    note_fills<kTma>(s, filled, true, warp, lane);
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
    finish4<D>(a, o, v, res, row, j);
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

// A persistent grid: as many pairs as the device holds at once (two blocks to
// a pair, one block to an SM), or fewer tiles.
template <int D, int kWord, bool kBoth, uint32_t kSubs, int kExtra>
cudaError_t launch_wide(const GemmArgs& a, const CUtensorMap (&m)[4], const SecondMaps<kExtra>& m2, int sms,
                        cudaStream_t st) {
  const uint32_t tiles = a.tiles_p * a.tiles_q, pairs = uint32_t(sms) / 2, rest = tiles % pairs;
  const bool halves = kSubs == 2 && 2 * rest <= pairs;
  GemmArgs g = a;
  g.whole = halves ? tiles - rest : tiles;
  g.pieces = halves ? tiles + rest : tiles;
  uint32_t smem = 1024 + g.stages * g.stage_bytes + kEpilogueWarps<kWord == 16> * kStagedBytes;
  if (smem < kAloneShared) smem = kAloneShared;
  return launch_cluster<gemm_wide_kernel<D, kWord, kBoth, kSubs, kExtra>>(2 * (g.pieces < pairs ? g.pieces : pairs),
                                                                       kGemmThreads<kWord == 16>, 2, smem, st, g, m[0],
                                                                       m[1], m[2], m[3], m2);
}

template <int D, int kWord, bool kBoth, int kExtra>
cudaError_t launch_split(const GemmArgs& a, const CUtensorMap (&m)[4], const SecondMaps<kExtra>& m2, cudaStream_t st) {
  return launch_cluster<gemm_split_kernel<D, kWord, kBoth, kExtra>>(a.tiles_p * a.tiles_q * a.split,
                                                                  kGemmThreads<kWord == 16>, a.split,
                                                                  1024 + a.stages * a.stage_bytes, st, a, m[0], m[1], m2);
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
      RealignSet r{};
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
  a.steps = a.first_steps = ceil_div(c.k, kStep);
  const bool sum = c.p2 && c.q2, stack = c.p2 && !c.q2;
  if (sum) a.steps *= 2;
  a.out2 = static_cast<uint16_t*>(c.out2), a.ldout2 = c.ldout2;

  const auto aligned = [](const void* p, uint64_t ld, unsigned elements) {
    return !p || (reinterpret_cast<uintptr_t>(p) % (2 * elements) == 0 && ld % elements == 0);
  };
  const auto out_aligned = [&](unsigned n) {
    return aligned(a.out, a.ldout, n) && aligned(a.z, a.ldz, n) && aligned(a.residual, a.ldresidual, n) &&
           aligned(a.out2, a.ldout2, n);
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
  const Tiles tiles = tiles_of(c, wide, a.bn, form.subs);
  a.tiles_p = wide ? tiles.rows : tiles.cols;
  a.tiles_q = wide ? tiles.cols : tiles.rows;
  a.tiles_first = tiles.rows / 2;  // of two stacked products
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
  SecondMaps<kSum> two{};
  SecondMaps<kStack> stacked{};
  if (c.p2) {
    if (word != 16) return cudaErrorInvalidValue;  // the caller brings all operands onto rows of 16 bytes
    // The layouts are those of the first operands: they go by the sizes.
    uint32_t layout;
    const auto* p2 = static_cast<const uint16_t*>(c.p2);
    const auto* q2 = static_cast<const uint16_t*>(c.q2);
    const auto second = [&](CUtensorMap* m, const uint16_t* base, uint64_t ld, bool is_p) {
      return is_p ? encode(m, &layout, base, ld, a.P, a.K, a.p_mn, kLanes, bf16)
                  : encode(m, &layout, base, ld, a.Q, a.K, a.q_mn, a.bq, bf16);
    };
    err = second(sum ? (wide ? &two.p : &two.q) : &stacked.in, p2, c.ldp2, wide);
    if (err == cudaSuccess && sum) err = second(wide ? &two.q : &two.p, q2, c.ldq2, !wide);
    if (err == cudaSuccess && stack && wide && a.octets)
      err = encode_output(&stacked.out, a.out2, a.ldout2, a.P, a.Q, bf16);
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
    const auto pairs = [&](const auto& second) {
      using M = std::remove_const_t<std::remove_reference_t<decltype(second)>>;
      constexpr int kExtra = std::is_same_v<M, SecondMaps<kSum>> ? kSum : std::is_same_v<M, SecondMaps<kStack>> ? kStack : kNone;
      if constexpr (kWord == 16)
        if (wide && form.subs == 2)
          return bf16 ? launch_wide<ARX_BF16, kWord, kBoth, 2, kExtra>(a, m, second, sms, st)
                      : launch_wide<ARX_F16, kWord, kBoth, 2, kExtra>(a, m, second, sms, st);
      if (wide)
        return bf16 ? launch_wide<ARX_BF16, kWord, kBoth, 1, kExtra>(a, m, second, sms, st)
                    : launch_wide<ARX_F16, kWord, kBoth, 1, kExtra>(a, m, second, sms, st);
      return bf16 ? launch_split<ARX_BF16, kWord, kBoth, kExtra>(a, m, second, st)
                  : launch_split<ARX_F16, kWord, kBoth, kExtra>(a, m, second, st);
    };
    if constexpr (kWord == 16) {
      if (sum) return pairs(two);
      if (stack) return pairs(stacked);
    }
    return pairs(SecondMaps<kNone>{});
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
