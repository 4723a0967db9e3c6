// Gated feed-forward block, forward: both projections, the activation and the
// product in one kernel.
//
// out[i][j] = act(g) u with g = sum_k x(i, k) Wg(j, k) and u with Wu: two
// products that share x.  A tile's accumulator holds g and u of the same
// elements side by side, so that the epilogue has both and neither goes to
// memory (unless the backward pass wants them).  Operands of 16 bits, or e4m3
// with scales of x's rows and the weights' rows, at twice the rate; a stage of
// the ring is 128 bytes of contraction either way.
//
// Three forms, chosen by estimates of their time (choose_gated_form; for one or two
// rows by sizes, dot_units):
//  vector one or two rows: dot products on the CUDA cores, a warp taking a
//         feature of both weights (one token, 4096 -> 2048: 6.0 us, 5.6 TB/s);
//  wide   persistent pairs of blocks.  The tensor cores' B operand is split over
//         the pair: the first block brings in rows of Wg, the second the same rows
//         of Wu, and an accumulator's first half is g, its second u (8185 tokens,
//         4096 -> 4096 bf16, both projections kept: 328 to 337 us, 1.6 PFLOP/s, and
//         e4m3, 1024 of 8192 -> 8192: 83 to 85 us, 3.3 PFLOP/s, while the card is
//         cool; back to back 343 and 96, bound by the card's power);
//  split  for few tokens: 64 features' rows of Wg and of Wu take the 128
//         accumulator lanes, the tokens the instruction's N, and a cluster of up to
//         8 blocks splits the contraction (e4m3, 32 of 8192 -> 4096: 15.3 us, of
//         which about 4 are the set-up and the join and the rest the weights' bytes).
// 16-bit operands off 16 bytes are copied to aligned rows first (realign.cu),
// but for one or two rows of small weights, which are read element by element.
#include <cuda_runtime.h>

#include "activation.cuh"
#include "gemm.cuh"

namespace arx {
namespace {

struct GatedArgs {
  GemmArgs g;  // P = tokens, Q = features of either weight (split: the other way around); bn: columns of an
               // accumulator (wide: bq = bn / 2 features); z: g, bias: its bias
  uint16_t* z_up;
  uint64_t ldz_up;
  const void* bias_up;
  const float *x_scale, *gate_scale, *up_scale;
  uint32_t k_step;  // contraction elements in a stage
};

// Features of a tile of the split form.
constexpr uint32_t kFeatures = kLanes / 2;

// ---- filling a stage ---------------------------------------------------------------

// One thread, a piece of kSubs accumulators; as copy_tile.
template <uint32_t kSubs>
__device__ __forceinline__ uint32_t copy_wide(const GatedArgs& a, const CUtensorMap* mx, const CUtensorMap* mw, Shared& s,
                                              uint8_t* stages, Ring& ring, uint32_t p0, uint32_t n0, uint32_t rank) {
  const uint32_t bytes = copied_bytes(a.g, kSubs);
  for (uint32_t i = 0; i < a.g.steps; ++i) {
    if (!mbar_wait(addr_of(&s.empty[ring.slot]), ring.phase ^ 1, &s.waits)) return i;
    const uint32_t dst = addr_of(stages + ring.slot * a.g.stage_bytes);
    uint32_t bar = addr_of(&s.full[ring.slot]);
    if (rank == 0) mbar_arrive_expect(bar, 2 * bytes);
    bar = cluster_peer_address(bar, 0);
    copy_box<true>(dst, mx, i * a.k_step, p0, bar);
#pragma unroll
    for (uint32_t j = 0; j < kSubs; ++j)
      copy_box<true>(dst + kPBytes + j * a.g.bq * 128, mw, i * a.k_step, n0 + j * a.g.bq, bar);
    ring.next(a.g.stages);
  }
  return a.g.steps;
}

__device__ __forceinline__ uint32_t copy_split(const GatedArgs& a, const CUtensorMap* mx, const CUtensorMap* mg,
                                               const CUtensorMap* mu, Shared& s, uint8_t* stages, Ring& ring, uint32_t n0,
                                               uint32_t m0, uint32_t first, uint32_t last) {
  const uint32_t bytes = copied_bytes(a.g, 1);
  for (uint32_t i = first; i < last; ++i) {
    if (!mbar_wait(addr_of(&s.empty[ring.slot]), ring.phase ^ 1, &s.waits)) return i - first;
    const uint32_t dst = addr_of(stages + ring.slot * a.g.stage_bytes), bar = addr_of(&s.full[ring.slot]);
    mbar_arrive_expect(bar, bytes);
    copy_box<false>(dst, mg, i * a.k_step, n0, bar);
    copy_box<false>(dst + kPBytes / 2, mu, i * a.k_step, n0, bar);
    copy_box<false>(dst + kPBytes, mx, i * a.k_step, m0, bar);
    ring.next(a.g.stages);
  }
  return last - first;
}

// ---- epilogues ------------------------------------------------------------------------

// Biases and scales of 32 columns from `col` on: asked for by the lanes a run of
// columns ahead, then put into shared memory, from where a warp reads four columns'
// at once.  (Handed round by shuffles they took an instruction for each column
// and vector: 128 of a run's 900 or so.)
struct Columns32 {
  float v[4];  // of this lane's column: bias_gate, bias_up, gate_scale, up_scale
};
__device__ __forceinline__ float ask_bias(const void* p, int wdtype, int D, uint32_t col, bool on) {
  on = on && p;
  if (wdtype == ARX_F32) return __uint_as_float(load_ahead4(static_cast<const float*>(p) + col, on));
  const uint16_t v = load_ahead2(static_cast<const uint16_t*>(p) + col, on);
  return D == ARX_BF16 ? Elem<ARX_BF16>::widen(v) : Elem<ARX_F16>::widen(v);
}
template <int D, bool k8>
__device__ __forceinline__ Columns32 ask_columns(const GatedArgs& a, uint32_t col, bool on) {
  on = on && col < a.g.Q;
  Columns32 c;
  c.v[0] = ask_bias(a.g.bias, a.g.wdtype, D, col, on);
  c.v[1] = ask_bias(a.bias_up, a.g.wdtype, D, col, on);
  c.v[2] = c.v[3] = 1.0f;
  if (k8) {
    if (a.gate_scale) c.v[2] = __uint_as_float(load_ahead4(a.gate_scale + col, on));
    if (a.up_scale) c.v[3] = __uint_as_float(load_ahead4(a.up_scale + col, on));
  }
  return c;
}

// Both projections' 32 columns: all loads on their way before the first wait.
__device__ __forceinline__ void load_sums(uint32_t gate, uint32_t up, bool any, float (&g)[32], float (&u)[32]) {
  uint32_t r[4][16];
  if (any) {
    tmem_load16_start(gate, r[0]);
    tmem_load16_start(gate + 16, r[1]);
    tmem_load16_start(up, r[2]);
    tmem_load16_start(up + 16, r[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) tmem_load_wait(r[i]);
  }
#pragma unroll
  for (int k = 0; k < 32; ++k) {
    g[k] = any ? __uint_as_float(r[k / 16][k % 16]) : 0.0f;
    u[k] = any ? __uint_as_float(r[2 + k / 16][k % 16]) : 0.0f;
  }
}

// v = v * scales + bias of 32 columns of this lane's row; the columns' at `bias`
// and `scale` in shared memory.
template <bool k8>
__device__ __forceinline__ void finish_sums(float (&v)[32], float row_scale, const float* scale, bool has_bias,
                                            const float* bias) {
#pragma unroll
  for (int k = 0; k < 32; k += 4) {
    Pair lo = pair(v[k], v[k + 1]), hi = pair(v[k + 2], v[k + 3]);
    if (k8) {
      const float4 f = *reinterpret_cast<const float4*>(scale + k);
      lo = lo * (pair(row_scale) * pair(f.x, f.y));
      hi = hi * (pair(row_scale) * pair(f.z, f.w));
    }
    if (has_bias) {
      const float4 f = *reinterpret_cast<const float4*>(bias + k);
      lo = lo + pair(f.x, f.y);
      hi = hi + pair(f.z, f.w);
    }
    halves(lo, v[k], v[k + 1]);
    halves(hi, v[k + 2], v[k + 3]);
  }
}

// As store_box, of the first 16 columns alone (rows of 32 bytes, not swizzled).
template <int D>
__device__ __forceinline__ void store_box16(const CUtensorMap* map, const float (&v)[32], uint32_t row0, uint32_t col,
                                            Boxes& boxes, uint32_t lane) {
  const uint32_t box = boxes.addr + boxes.turn * 2048;
  boxes.turn ^= 1;
  if (lane == 0) bulk_wait_read<1>();  // the box's last store has read it
  __syncwarp();
#pragma unroll
  for (uint32_t u = 0; u < 2; ++u) {
    uint32_t w[4];
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) w[i] = Elem<D>::round2(v[8 * u + 2 * i], v[8 * u + 2 * i + 1]);
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                 :: "r"(box + lane * 32 + u * 16), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
  }
  fence_async_shared();
  __syncwarp();
  if (lane == 0) tma_store_2d(map, col, row0, box);
}

// Rows off 16 bytes: 32 rows by 32 columns staged in shared memory as [row][33];
// a lane takes a column and walks down the rows, so that the warp stores a row's
// line at a time.
template <int D>
__device__ __forceinline__ void store_staged(float* staged, const float (&v)[32], uint16_t* out, uint64_t ld, uint32_t rows,
                                             uint32_t row0, uint32_t col, uint32_t cols, uint32_t lane) {
  __syncwarp();
#pragma unroll
  for (uint32_t k = 0; k < 32; ++k) staged[lane * 33 + k] = v[k];
  __syncwarp();
  const uint32_t n = row0 < rows ? (rows - row0 < 32 ? rows - row0 : 32) : 0;
  if (col + lane >= cols) return;
  uint16_t* p = out + row0 * ld + col + lane;
#pragma unroll 8
  for (uint32_t r = 0; r < n; ++r, p += ld) *p = Elem<D>::round(staged[r * 33 + lane]);
}

// 32 rows by n columns of the outputs, by a warp.
__device__ __noinline__ void fill_outputs_nan(const GatedArgs& a, uint32_t row0, uint32_t col0, uint32_t n, uint32_t lane) {
  constexpr uint16_t kNan = 0x7FFF;  // in bf16 and in fp16
  for (uint64_t row = row0; row < row0 + 32 && row < a.g.P; ++row)
    for (uint32_t c = col0 + lane; c < col0 + n && c < a.g.Q; c += 32) {
      a.g.out[row * a.g.ldout + c] = kNan;
      if (a.g.z) a.g.z[row * a.g.ldz + c] = kNan;
      if (a.z_up) a.z_up[row * a.ldz_up + c] = kNan;
    }
}

// A warp's features of an accumulator: `width` from c0 on, a multiple of 16, in
// runs of 32 and at the end perhaps 16.
struct Share {
  uint32_t c0, width;
  __device__ __forceinline__ uint32_t runs() const { return (width + 31) / 32; }
};
__device__ __forceinline__ Share share_of(const GemmArgs& a, uint32_t warp) {
  const uint32_t first = (a.bq / 2 + 15) / 16 * 16;
  return warp < 6 ? Share{0, first} : Share{first, a.bq - first};
}

struct OutputMaps {
  CUtensorMap out, z_gate, z_up;
};

// D: type of the outputs (and of 16-bit operands); kSubs: accumulators to a tile.
template <int D, bool k8, uint32_t kSubs>
__global__ void __launch_bounds__(kGemmThreads<true>, 1)
    gated_wide_kernel(const __grid_constant__ GatedArgs args, const __grid_constant__ CUtensorMap mx,
                      const __grid_constant__ CUtensorMap mg, const __grid_constant__ CUtensorMap mu,
                      const __grid_constant__ OutputMaps m32, const __grid_constant__ OutputMaps m16) {
  const GemmArgs& a = args.g;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared s;
  uint8_t* stages = smem_raw + ((1024u - (addr_of(smem_raw) & 1023u)) & 1023u);
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x & 31, rank = cluster_ctarank();
  const CUtensorMap* mw = rank ? &mu : &mg;
  setup<true, true>(a, &mx, mw, s, warp);
  dependent_launch_prologue();
  const uint32_t pieces = a.pieces, first_piece = blockIdx.x / 2, step = gridDim.x / 2;

  Ring ring;
  if (threadIdx.x == 0) {
    uint32_t t = first_piece, filled = 0;
    for (; t < pieces; t += step) {
      const Piece w = piece_at<kSubs>(a, t);
      const uint32_t p0 = (2 * w.tp + rank) * kLanes, n0 = w.q0 / 2;
      filled = kSubs == 2 && w.subs == 2 ? copy_wide<kSubs>(args, &mx, mw, s, stages, ring, p0, n0, rank)
                                         : copy_wide<1>(args, &mx, mw, s, stages, ring, p0, n0, rank);
      if (filled < a.steps) break;
    }
    note_fills<true>(s, (t - first_piece) / step * a.steps + (t < pieces ? filled : 0), true, warp, lane);
  } else if (warp == 1 && lane == 0 && rank == 0 && a.steps > 0) {
    uint32_t n = 0;
    for (uint32_t t = first_piece; t < pieces; t += step, ++n) {
      const uint32_t b = kSubs == 2 ? 0 : n & 1, use = kSubs == 2 ? n : n >> 1;
      if (!mbar_wait(addr_of(&s.acc_empty[b]), (use & 1) ^ 1, &s.waits)) break;
      tmem_fence_after();
      const uint32_t subs = piece_at<kSubs>(a, t).subs;
      if (!(kSubs == 2 && subs == 2
                ? multiply_tile<true, kSubs, k8>(a, s, addr_of(stages), ring, s.tmem, 0, a.steps)
                : multiply_tile<true, 1, k8>(a, s, addr_of(stages), ring, s.tmem + b * 256, 0, a.steps)))
        break;
      mma_commit<true>(addr_of(&s.acc_full[b]));
    }
  } else if (warp >= 2) {
    const uint32_t quarter = warp & 3;  // the accumulator lanes this warp may read
    const Share share = share_of(a, warp);
    float* staged = reinterpret_cast<float*>(stages + a.stages * a.stage_bytes) + (warp - 2) * 32 * 33;
    Boxes boxes{addr_of(stages + a.stages * a.stage_bytes) + (warp - 2) * 4096, 0};
    uint8_t* const box0 = stages + a.stages * a.stage_bytes + (warp - 2) * 4096;
    uint32_t n = 0, t = first_piece;
    for (; t < pieces; t += step, ++n) {
      const Piece w = piece_at<kSubs>(a, t);
      const uint32_t b = kSubs == 2 ? 0 : n & 1, use = kSubs == 2 ? n : n >> 1;
      const uint32_t row0 = (2 * w.tp + rank) * kLanes + quarter * 32, n0 = w.q0 / 2;
      const uint32_t per = share.runs(), runs = row0 < a.P ? w.subs * per : 0;
      const auto column = [&](uint32_t i) { return n0 + i / per * a.bq + share.c0 + i % per * 32; };
      Columns32 ahead = ask_columns<D, k8>(args, column(0) + lane, runs > 0);
      float row_scale = 1.0f;
      if (k8 && args.x_scale) row_scale = __uint_as_float(load_ahead4(args.x_scale + row0 + lane, row0 + lane < a.P));
      if (a.steps > 0) {
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(addr_of(&s.acc_full[b]), use & 1, &s.waits))) break;
        tmem_fence_after();
      }
      for (uint32_t i = 0; i < runs; ++i) {
        const uint32_t col = column(i), j = i / per;
        if (col >= a.Q) break;  // and so are those after it
        const uint32_t wide = share.width - i % per * 32;  // 16, or 32 and more
        const uint32_t acc = s.tmem + (b + j) * 256 + (quarter * 32 << 16) + (col - n0 - j * a.bq);
        float g[32], u[32];
        load_sums(acc, acc + a.bq, a.steps > 0, g, u);
        if (k8 || a.bias || args.bias_up) {
          // In the box (or staging rows) that the run's first store takes afterwards.
          float(*own)[32] = reinterpret_cast<float(*)[32]>(a.octets ? box0 + boxes.turn * 2048 : reinterpret_cast<uint8_t*>(staged));
          if (lane == 0) bulk_wait_read<1>();
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 4; ++k) own[k][lane] = ahead.v[k];
          __syncwarp();
          ahead = ask_columns<D, k8>(args, column(i + 1) + lane, i + 1 < runs);
          finish_sums<k8>(g, row_scale, own[2], a.bias != nullptr, own[0]);
          finish_sums<k8>(u, row_scale, own[3], args.bias_up != nullptr, own[1]);
        }
        const auto store = [&](const CUtensorMap* map32, const CUtensorMap* map16, const float(&v)[32], uint16_t* p,
                               uint64_t ld) {
          if (!a.octets)
            store_staged<D>(staged, v, p, ld, a.P, row0, col, wide < 32 && col + 16 < a.Q ? col + 16 : a.Q, lane);
          else if (wide < 32)
            store_box16<D>(map16, v, row0, col, boxes, lane);
          else
            store_box<D>(map32, v, row0, col, boxes, lane);
        };
        if (a.z) store(&m32.z_gate, &m16.z_gate, g, a.z, a.ldz);
        if (args.z_up) store(&m32.z_up, &m16.z_up, u, args.z_up, args.ldz_up);
        activate<32>(g, a.act);
#pragma unroll
        for (int k = 0; k < 32; k += 2) halves(pair(g[k], g[k + 1]) * pair(u[k], u[k + 1]), g[k], g[k + 1]);
        store(&m32.out, &m16.out, g, a.out, a.ldout);
      }
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(cluster_peer_address(addr_of(&s.acc_empty[b]), 0));
    }
    for (; t < pieces; t += step) {  // after a wait ran out
      const Piece w = piece_at<kSubs>(a, t);
      for (uint32_t j = 0; j < w.subs; ++j)
        fill_outputs_nan(args, (2 * w.tp + rank) * kLanes + quarter * 32, w.q0 / 2 + j * a.bq + share.c0, share.width, lane);
    }
    if (lane == 0) bulk_wait_all();
  }
  __syncwarp();
  finish_block<true, true, kSubs>(a, s, warp, rank);
}

// Four consecutive features of a token.
template <int D>
__device__ __forceinline__ void store4(uint16_t* p, const float (&v)[4], bool whole, uint32_t n) {
  const uint2 w = make_uint2(Elem<D>::round2(v[0], v[1]), Elem<D>::round2(v[2], v[3]));
  if (whole) {
    st_global(reinterpret_cast<uint2*>(p), w);
  } else {
    const uint32_t h[4] = {w.x & 0xFFFFu, w.x >> 16, w.y & 0xFFFFu, w.y >> 16};
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k)
      if (k < n) p[k] = uint16_t(h[k]);
  }
}

// One tile per cluster; block r of the cluster takes the r-th share of the
// contraction.  P's rows are the features here, Q's rows the tokens.
template <int D, bool k8>
__global__ void __launch_bounds__(kGemmThreads<true>, 2)
    gated_split_kernel(const __grid_constant__ GatedArgs args, const __grid_constant__ CUtensorMap mx,
                       const __grid_constant__ CUtensorMap mg, const __grid_constant__ CUtensorMap mu) {
  const GemmArgs& a = args.g;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared s;
  uint8_t* stages = smem_raw + ((1024u - (addr_of(smem_raw) & 1023u)) & 1023u);
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  setup<true, false>(a, &mg, &mu, s, warp);
  dependent_launch_prologue();
  const uint32_t rank = blockIdx.x % a.split, tile = blockIdx.x / a.split;
  const uint32_t n0 = tile % a.tiles_p * kFeatures, m0 = tile / a.tiles_p * a.bn;
  const uint32_t share = (a.steps + a.split - 1) / a.split;
  const uint32_t first = rank * share < a.steps ? rank * share : a.steps;
  const uint32_t last = first + share < a.steps ? first + share : a.steps;
  float* part = reinterpret_cast<float*>(stages);  // [bn][128 lanes], once the stages are done with

  Ring ring;
  if (threadIdx.x == 0) {
    note_fills<true>(s, copy_split(args, &mx, &mg, &mu, s, stages, ring, n0, m0, first, last), true, warp, lane);
  } else if (warp == 1 && lane == 0 && first < last) {
    if (multiply_tile<false, 1, k8>(a, s, addr_of(stages), ring, s.tmem, first, last))
      mma_commit<false>(addr_of(&s.acc_full[0]));
  } else if (warp >= 2) {
    const uint32_t quarter = warp & 3;
    bool ok = true;
    if (first < last) {
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(addr_of(&s.acc_full[0]), 0, &s.waits));
      tmem_fence_after();
    }
    if (ok)
      for (uint32_t c = (warp - 2) / 4 * 16; c < a.bn; c += 32) {
        float v[16] = {};
        if (first < last) tmem_load16(s.tmem + c + (quarter * 32 << 16), v);
#pragma unroll
        for (int k = 0; k < 16; ++k) part[(c + k) * kLanes + quarter * 32 + lane] = v[k];
      }
  }
  __syncthreads();
  if (s.waits.abort) {  // its part of every sum is NaN, once nothing lands on it any more
    drain_block<true, false, 1>(a, s);
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < a.bn * kLanes; i += kGemmThreads<true>) part[i] = __int_as_float(0x7FFFFFFF);
    __syncthreads();
  }
  cluster_arrive_release();
  cluster_wait();

  // The tile's elements are shared out over the cluster's blocks in groups of
  // four features of a token; each sum is that of the partials in block order.
  const uint32_t tokens = a.Q - m0 < a.bn ? a.Q - m0 : a.bn;
  const uint32_t groups = tokens * (kFeatures / 4);
  const uint32_t per = (groups + a.split - 1) / a.split;
  const uint32_t end = (rank + 1) * per < groups ? (rank + 1) * per : groups;
  const uint32_t base = addr_of(part);
  for (uint32_t i = rank * per + threadIdx.x; i < end; i += kGemmThreads<true>) {
    const uint32_t f = i % (kFeatures / 4) * 4, token = i / (kFeatures / 4), j = n0 + f, row = m0 + token;
    const uint32_t at = base + (token * kLanes + f) * 4;
    const auto sum = [&](uint32_t from, float(&v)[4]) {
      float4 in[8];
#pragma unroll
      for (uint32_t r = 0; r < 8; ++r)
        if (r < a.split) in[r] = ld_cluster_f32x4(cluster_peer_address(from, r));
      v[0] = v[1] = v[2] = v[3] = 0.0f;
#pragma unroll
      for (uint32_t r = 0; r < 8; ++r)
        if (r < a.split) v[0] += in[r].x, v[1] += in[r].y, v[2] += in[r].z, v[3] += in[r].w;
    };
    if (j >= a.P) continue;
    const uint32_t n = a.P - j < 4 ? a.P - j : 4;
    float g[4], u[4];
    sum(at, g);
    sum(at + kFeatures * 4, u);
    if (k8) {
      const float sx = args.x_scale ? args.x_scale[row] : 1.0f;
#pragma unroll
      for (uint32_t k = 0; k < 4; ++k)
        if (k < n) {
          g[k] *= sx * (args.gate_scale ? args.gate_scale[j + k] : 1.0f);
          u[k] *= sx * (args.up_scale ? args.up_scale[j + k] : 1.0f);
        }
    }
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k) {
      if (a.bias && k < n) g[k] += load_param(a.bias, a.wdtype, j + k);
      if (args.bias_up && k < n) u[k] += load_param(args.bias_up, a.wdtype, j + k);
    }
    const bool whole = a.quads && n == 4;
    if (a.z) store4<D>(a.z + row * a.ldz + j, g, whole, n);
    if (args.z_up) store4<D>(args.z_up + row * args.ldz_up + j, u, whole, n);
    activate<4>(g, a.act);
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k) g[k] *= u[k];
    store4<D>(a.out + row * a.ldout + j, g, whole, n);
  }
  finish_block<true, false, 1>(a, s, warp, rank);
}

// ---- one or two rows --------------------------------------------------------------------
//
// Both weights are read once, which bounds the kernel.  A warp (or `split` warps
// of a block) takes a feature: its lanes take 16-byte units of the feature's two
// rows, kDotBatch of each in flight, and x comes from L1.  The lanes' sums meet in
// a butterfly and the split warps' in warp order.  kV = 1: rows off 16 bytes,
// element by element.

constexpr uint32_t kDotRows = 2;
constexpr uint32_t kDotThreads = 256;
constexpr int kDotBatch = 4;  // 2 took 1.0 to 1.25 times as long, 8 1.2 to 1.5 (fewer blocks at once)

// Two e4m3 in 16 bits, widened.
__device__ __forceinline__ void widen_e4m3x2(uint32_t v, float& a, float& b) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(v)));
  Elem<ARX_F16>::widen2(h, a, b);
}

template <int I, int kV>  // kV elements of an operand of type I: 16 bytes, or one
struct Unit;
template <int I>
struct Unit<I, 8> {
  uint4 w;
  __device__ __forceinline__ void get(float (&f)[8]) const {
    Elem<I>::widen2(w.x, f[0], f[1]);
    Elem<I>::widen2(w.y, f[2], f[3]);
    Elem<I>::widen2(w.z, f[4], f[5]);
    Elem<I>::widen2(w.w, f[6], f[7]);
  }
};
template <>
struct Unit<ARX_E4M3, 16> {
  uint4 w;
  __device__ __forceinline__ void get(float (&f)[16]) const {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      widen_e4m3x2(v[i] & 0xFFFFu, f[4 * i], f[4 * i + 1]);
      widen_e4m3x2(v[i] >> 16, f[4 * i + 2], f[4 * i + 3]);
    }
  }
};
template <int I>
struct Unit<I, 1> {
  uint16_t w;
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = Elem<I>::widen(w); }
};

template <int I, int O, int kM, int kV>
__global__ void __launch_bounds__(kDotThreads) gated_dot_kernel(const __grid_constant__ GatedArgs args, const void* w_up,
                                                                uint64_t ldw_up) {
  constexpr uint32_t kSize = I == ARX_E4M3 ? 1 : 2;
  using Word = decltype(Unit<I, kV>::w);
  const GemmArgs& a = args.g;
  __shared__ float part[kDotThreads / 32][2 * kM];
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const uint32_t per = kDotThreads / 32 / a.split;  // features of a block
  const uint32_t j = blockIdx.x * per + warp / a.split, share = warp % a.split;
  const uint8_t* row[2] = {reinterpret_cast<const uint8_t*>(a.q) + j * a.ldq * kSize,
                           static_cast<const uint8_t*>(w_up) + j * ldw_up * kSize};
  // A hint only, as in linear.cu: the weights' way to L2 starts while the stream's
  // previous kernel, whose output x may be, still runs.  The first batch of the
  // feature's warps: asked for whole, rows of 16 KB came twice (8192 x 8192: 55.8
  // against 44.5 us; none 44.9, but 2048 x 4096 7.3 against 6.2).
  if (kV > 1 && share == 0 && lane == 0 && j < a.Q && a.K > 0) {
    const uint32_t bytes = a.K * kSize, batch = 32 * kDotBatch * 16 * a.split;
    for (int h = 0; h < 2; ++h) prefetch_l2_bulk(row[h], bytes < batch ? bytes : batch);
  }
  dependent_launch_prologue();
  float acc[2 * kM] = {};
  if (j < a.Q) {
    const uint32_t units = a.K / kV, step = 32 * a.split;
    for (uint32_t u0 = share * 32 + lane; u0 < units; u0 += kDotBatch * step) {
      Unit<I, kV> wv[2][kDotBatch];
#pragma unroll
      for (int b = 0; b < kDotBatch; ++b)
        if (u0 + b * step < units)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const Word* p = reinterpret_cast<const Word*>(row[h]) + u0 + b * step;
            if constexpr (kV == 1)
              wv[h][b].w = *p;
            else
              wv[h][b].w = ld_stream(p);
          }
#pragma unroll
      for (int b = 0; b < kDotBatch; ++b) {
        if (u0 + b * step >= units) break;
        float f[2][kV];
        wv[0][b].get(f[0]);
        wv[1][b].get(f[1]);
#pragma unroll
        for (int m = 0; m < kM; ++m) {
          Unit<I, kV> xv;
          xv.w = reinterpret_cast<const Word*>(reinterpret_cast<const uint8_t*>(a.p) + m * a.ldp * kSize)[u0 + b * step];
          float x[kV];
          xv.get(x);
#pragma unroll
          for (int k = 0; k < kV; ++k) {
            acc[2 * m] = fmaf(f[0][k], x[k], acc[2 * m]);
            acc[2 * m + 1] = fmaf(f[1][k], x[k], acc[2 * m + 1]);
          }
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 2 * kM; ++i) acc[i] = warp_sum(acc[i]);
  if (a.split > 1) {
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < 2 * kM; ++i) part[warp][i] = acc[i];
    __syncthreads();
    if (share == 0)
      for (uint32_t r = 1; r < a.split; ++r)
#pragma unroll
        for (int i = 0; i < 2 * kM; ++i) acc[i] += part[warp + r][i];
  }
  if (share != 0 || j >= a.Q) return;
#pragma unroll
  for (int m = 0; m < kM; ++m)
    if (lane == uint32_t(m)) {
      float g[1] = {acc[2 * m]}, u = acc[2 * m + 1];
      if (I == ARX_E4M3) {
        const float sx = args.x_scale ? args.x_scale[m] : 1.0f;
        g[0] *= sx * (args.gate_scale ? args.gate_scale[j] : 1.0f);
        u *= sx * (args.up_scale ? args.up_scale[j] : 1.0f);
      }
      if (a.bias) g[0] += load_param(a.bias, a.wdtype, j);
      if (args.bias_up) u += load_param(args.bias_up, a.wdtype, j);
      if (a.z) a.z[m * a.ldz + j] = Elem<O>::round(g[0]);
      if (args.z_up) args.z_up[m * args.ldz_up + j] = Elem<O>::round(u);
      activate<1>(g, a.act);
      a.out[m * a.ldout + j] = Elem<O>::round(g[0] * u);
    }
}

// ---- host side ---------------------------------------------------------------------

// Map of an operand of `rows` by `k`, for boxes of `tile` rows by 128 bytes.
cudaError_t encode_rows(CUtensorMap* m, const void* base, uint64_t ld, uint64_t rows, uint64_t k, uint32_t tile, int dtype) {
  cudaError_t err = cudaSuccess;
  auto f = encode_function(&err);
  if (!f) return err;
  const uint64_t size = dtype == ARX_E4M3 ? 1 : 2;
  const cuuint64_t dims[2] = {k, rows}, strides[1] = {rows > 1 ? ld * size : (k * size + 15) / 16 * 16};
  const cuuint32_t box[2] = {cuuint32_t(128 / size), tile}, el[2] = {1, 1};
  const CUtensorMapDataType type = dtype == ARX_E4M3   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : dtype == ARX_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                       : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const CUresult r = f(m, type, 2, const_cast<void*>(base), dims, strides, box, el, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

bool on_16_bytes(const void* p, uint64_t ld, uint64_t rows, uint64_t size) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows <= 1 || ld * size % 16 == 0);
}

uint64_t size_of(int dtype) { return dtype == ARX_E4M3 ? 1 : 2; }

// Do dot products take the call in whole units?  Measured, microseconds (dot, split
// form): one row, 16 bits, 2048 x 4096 6.2, 9.4; 4096 x 8192 21.6, 23.3; 8192 x 8192
// 43.9, 41.9; e4m3 the dot form up to there.  Two rows, whose second halves the
// reading's share of the issue slots, 4096 x 4096 13.0, 13.9; 4096 x 8192 25.0, 23.4;
// e4m3, with its conversions, 512 x 1024 2.4, 4.3; 1024 x 2048 4.7, 4.6; 4096 x 8192
// 21.3, 14.7.
bool dot_units(const arx_gated_linear_args& c) {
  const uint64_t size = size_of(c.dtype), weights = 2 * c.N * c.K;
  if (c.M > kDotRows) return false;
  if (c.dtype == ARX_E4M3 ? c.M == 2 && weights > (1u << 22) : weights >= (c.M == 2 ? 3u << 24 : 1u << 27)) return false;
  return c.K * size % 16 == 0 && on_16_bytes(c.x, c.ldx, c.M, size) &&
         on_16_bytes(c.w_gate, c.ldw_gate, c.N, size) && on_16_bytes(c.w_up, c.ldw_up, c.N, size);
}
// One by one (16 bits)?  As the products of linear.cu: up to about 8 million weights.
bool dot_single(const arx_gated_linear_args& c) {
  return c.M <= kDotRows && c.dtype != ARX_E4M3 && 2 * c.N * c.K < (uint64_t(1) << 23);
}

// The operands to be copied onto rows of 16 bytes, in the order x, w_gate, w_up.
struct GatedCopies {
  bool on[3];
  uint64_t bytes[3], total;
};
GatedCopies copies_of(const arx_gated_linear_args& c) {
  GatedCopies r{};
  if (c.M == 0 || c.N == 0 || c.K == 0 || c.dtype == ARX_E4M3 || dot_units(c) || dot_single(c)) return r;
  const void* p[3] = {c.x, c.w_gate, c.w_up};
  const uint64_t ld[3] = {c.ldx, c.ldw_gate, c.ldw_up}, rows[3] = {c.M, c.N, c.N};
  for (int i = 0; i < 3; ++i) {
    r.on[i] = !on_16_bytes(p[i], ld[i], rows[i], 2);
    r.bytes[i] = r.on[i] ? rows[i] * ((c.K + 7) / 8 * 16) : 0;
    r.total += r.bytes[i];
  }
  return r;
}

// The split form's estimate is choose_form's, with 20 cycles more for a token that a
// block of 256 stores alone (both sums and the activation, and no second block on the
// SM to work meanwhile; e4m3 [512, 1024] x [1024, 4096]: 20.2 us, the wide form 10.1)
// and a part of it where a cluster shares them.  The wide form's tiles are 64 to 128
// features (bn / 2) to an accumulator, so that the last round of tiles is full: of
// e4m3 [1024, 8192] x [8192, 8192], two accumulators, 152 pairs of tiles in two
// rounds of 76 take 91.7 us with 128 features, and 148 of 112 84.4 (one
// accumulator, four rounds: 90.1, 89.0).  Measured, cycles of a stage: 600
// for one accumulator of 256 columns, bound by the copies (55 bytes a cycle into
// an SM, more while few pairs are at work and less for the shorter copies of narrow
// tiles), 580 for one of 224; 4.25 a column of two, bound by the products (4.2).
// What is outside the stages: with one accumulator 10500 (256 tokens of 64 -> 4096: 5.9
// us) and, until the rings are full, up to 5500 when all pairs ask at once; 12500 for
// a round with two, whose epilogue no products hide; and 2900 for each projection that
// is kept.
Form choose_gated_form(const arx_gated_linear_args& c, uint32_t steps) {
  GemmCall shape{};
  shape.rows = c.M, shape.cols = 2 * c.N, shape.k = c.K;
  Form best = choose_form(shape, steps, true, true, false, 20);
  constexpr uint32_t pairs = 152 / 2;
  const double kept = 2900.0 * ((c.z_gate != nullptr) + (c.z_up != nullptr));
  best.cycles += kept;
  for (uint32_t bn = 256; bn >= 128; bn -= 32)
    for (uint32_t subs = 1; subs <= 2; ++subs) {
      const uint32_t tiles = ceil_div(c.M, 2 * kLanes) * ceil_div(c.N, subs * bn / 2), rest = tiles % pairs;
      const double at_work = double(tiles < pairs ? tiles : pairs) / pairs;
      const double engine = bn >= 224 ? 64 - 10 * at_work : bn >= 192 ? 54 : 46;
      const double copies = (kLanes + bn / 2) * 128.0 / engine, one = copies > 2.1 * bn ? copies : 2.1 * bn;
      double cycles;
      if (subs == 1) {
        const double tile = steps * one, epilogue = 4000 + kept;
        const double fill = steps < 6 ? steps / 6.0 : 1;
        cycles = tile + (ceil_div(tiles, pairs) - 1) * (tile > epilogue ? tile : epilogue) + 10500 +
                 5500 * at_work * fill + kept;
      } else {
        const double all = (kLanes + bn) * 128.0 / 46, two = all > 4.25 * bn ? all : 4.25 * bn;
        const bool halves = rest && 2 * rest <= pairs;
        cycles = (tiles / pairs + (rest && !halves)) * (steps * two + 12500 + kept) +
                 (halves ? steps * one * 1.25 + 8000 + kept : 0) + 11000;
      }
      if (cycles < best.cycles) best = {true, bn, 1, subs, tiles, cycles};
    }
  return best;
}

template <int I, int O, int kV>
cudaError_t launch_dot(const GatedArgs& a, const void* w_up, uint64_t ldw_up, cudaStream_t st) {
  const dim3 grid(ceil_div(a.g.Q, kDotThreads / 32 / a.g.split));
  return a.g.P == 1 ? launch_op(gated_dot_kernel<I, O, 1, kV>, grid, kDotThreads, 0, st, a, w_up, ldw_up)
                    : launch_op(gated_dot_kernel<I, O, 2, kV>, grid, kDotThreads, 0, st, a, w_up, ldw_up);
}

template <int D, bool k8, uint32_t kSubs>
cudaError_t launch_wide(const GatedArgs& a, const CUtensorMap (&m)[3], const OutputMaps (&o)[2], int sms,
                        cudaStream_t st) {
  const uint32_t tiles = a.g.tiles_p * a.g.tiles_q, pairs = uint32_t(sms) / 2, rest = tiles % pairs;
  const bool halves = kSubs == 2 && 2 * rest <= pairs;
  GatedArgs b = a;
  b.g.whole = halves ? tiles - rest : tiles;
  b.g.pieces = halves ? tiles + rest : tiles;
  uint32_t smem = 1024 + b.g.stages * b.g.stage_bytes + kEpilogueWarps<true> * kStagedBytes;
  if (smem < kAloneShared) smem = kAloneShared;
  return launch_cluster<gated_wide_kernel<D, k8, kSubs>>(2 * (b.g.pieces < pairs ? b.g.pieces : pairs),
                                                        kGemmThreads<true>, 2, smem, st, b, m[0], m[1], m[2], o[0], o[1]);
}

template <int D, bool k8>
cudaError_t launch_split(const GatedArgs& a, const CUtensorMap (&m)[3], cudaStream_t st) {
  return launch_cluster<gated_split_kernel<D, k8>>(a.g.tiles_p * a.g.tiles_q * a.g.split, kGemmThreads<true>, a.g.split,
                                                   1024 + a.g.stages * a.g.stage_bytes, st, a, m[0], m[1], m[2]);
}

}  // namespace

size_t gated_copies_bytes(const arx_gated_linear_args& c) { return size_t(copies_of(c).total); }

cudaError_t launch_gated(const arx_gated_linear_args& c, cudaStream_t st) {
  cudaError_t err = cudaSuccess;
  const GatedCopies copies = copies_of(c);
  if (copies.total) {
    arx_gated_linear_args on = c;
    const void** p[3] = {&on.x, &on.w_gate, &on.w_up};
    uint64_t* ld[3] = {&on.ldx, &on.ldw_gate, &on.ldw_up};
    const uint64_t rows[3] = {c.M, c.N, c.N};
    RealignSet r{};
    uint8_t* dst = static_cast<uint8_t*>(c.copies);
    for (int i = 0; i < 3; ++i) {
      if (!copies.on[i]) continue;
      const uint64_t pitch = (c.K + 7) / 8 * 8;
      r.m[r.n++] = {static_cast<const uint16_t*>(*p[i]), reinterpret_cast<uint16_t*>(dst), rows[i], *ld[i], pitch,
                    int64_t(c.K)};
      *p[i] = dst, *ld[i] = pitch;
      dst += copies.bytes[i];
    }
    err = launch_realign(r, st);
    return err != cudaSuccess ? err : launch_gated(on, st);
  }
  const int sms = current_sm_count(&err);
  if (sms < 1) return err;
  const bool k8 = c.dtype == ARX_E4M3, bf16 = c.out_dtype == ARX_BF16;
  GatedArgs a{};
  GemmArgs& g = a.g;
  g.out = static_cast<uint16_t*>(c.out), g.ldout = c.ldout;
  g.z = static_cast<uint16_t*>(c.z_gate), g.ldz = c.ldz_gate;
  a.z_up = static_cast<uint16_t*>(c.z_up), a.ldz_up = c.ldz_up;
  g.bias = c.bias_gate, a.bias_up = c.bias_up;
  a.x_scale = c.x_scale, a.gate_scale = c.gate_scale, a.up_scale = c.up_scale;
  g.status = c.status;
  g.wait_ns = uint32_t(c.wait_us) * 1000u;
  g.act = c.act, g.wdtype = c.wdtype;
  g.K = uint32_t(c.K);
  a.k_step = k8 ? 128 : 64;
  g.steps = ceil_div(c.K, a.k_step);

  const bool units = dot_units(c);
  if (units || dot_single(c)) {
    g.p = static_cast<const uint16_t*>(c.x), g.ldp = c.ldx;
    g.q = static_cast<const uint16_t*>(c.w_gate), g.ldq = c.ldw_gate;
    g.P = uint32_t(c.M), g.Q = uint32_t(c.N);
    // Warps for about 16 to an SM, while each keeps 256 elements or more.
    g.split = 1;
    while (g.split < 8 && uint64_t(g.Q) * g.split < 2432 && g.K / g.split > 512) g.split *= 2;
    if (k8)
      return bf16 ? launch_dot<ARX_E4M3, ARX_BF16, 16>(a, c.w_up, c.ldw_up, st)
                  : launch_dot<ARX_E4M3, ARX_F16, 16>(a, c.w_up, c.ldw_up, st);
    if (bf16)
      return units ? launch_dot<ARX_BF16, ARX_BF16, 8>(a, c.w_up, c.ldw_up, st)
                   : launch_dot<ARX_BF16, ARX_BF16, 1>(a, c.w_up, c.ldw_up, st);
    return units ? launch_dot<ARX_F16, ARX_F16, 8>(a, c.w_up, c.ldw_up, st)
                 : launch_dot<ARX_F16, ARX_F16, 1>(a, c.w_up, c.ldw_up, st);
  }

  const auto aligned = [](const void* p, uint64_t ld, unsigned elements) {
    return !p || (reinterpret_cast<uintptr_t>(p) % (2 * elements) == 0 && ld % elements == 0);
  };
  const auto out_aligned = [&](unsigned n) {
    return aligned(c.out, c.ldout, n) && aligned(c.z_gate, c.ldz_gate, n) && aligned(c.z_up, c.ldz_up, n);
  };
  g.quads = out_aligned(4);
  g.octets = out_aligned(8) && c.N % 8 == 0;

  const Form form = choose_gated_form(c, g.steps);
  g.bn = form.bn, g.split = form.split;
  g.p_copy = g.q_copy = c.K > 0;
  if (form.wide) {
    g.P = uint32_t(c.M), g.Q = uint32_t(c.N);
    g.bq = g.bn / 2;
    g.tmem_columns = 512;
    g.tiles_p = ceil_div(g.P, 2 * kLanes);
    g.tiles_q = ceil_div(g.Q, form.subs * g.bq);
  } else {
    g.P = uint32_t(c.N), g.Q = uint32_t(c.M);
    g.bq = g.bn;
    g.tmem_columns = g.bn < 32 ? 32 : g.bn;
    g.tiles_p = ceil_div(g.P, kFeatures);
    g.tiles_q = ceil_div(g.Q, g.bn);
  }
  g.stage_bytes = kPBytes + form.subs * g.bq * 128;
  g.stages = (form.wide || g.bn > 128 ? kStageBudget : kSplitBudget) / g.stage_bytes;
  if (g.stages > kMaxStages) g.stages = kMaxStages;
  g.idesc = mma_descriptor(c.dtype == ARX_BF16, false, false, form.wide ? 2 * kLanes : kLanes, g.bn);

  CUtensorMap m[3] = {};  // x, w_gate, w_up
  OutputMaps o[2] = {};   // boxes of 32 columns and of 16
  if (c.K > 0) {
    const uint32_t w_tile = form.wide ? g.bq : kFeatures;
    err = encode_rows(&m[0], c.x, c.ldx, c.M, c.K, form.wide ? kLanes : g.bn, c.dtype);
    if (err == cudaSuccess) err = encode_rows(&m[1], c.w_gate, c.ldw_gate, c.N, c.K, w_tile, c.dtype);
    if (err == cudaSuccess) err = encode_rows(&m[2], c.w_up, c.ldw_up, c.N, c.K, w_tile, c.dtype);
    if (err != cudaSuccess) return err;
  }
  if (form.wide && g.octets)
    for (int i = 0; i < 2; ++i) {
      const uint32_t columns = i ? 16 : 32;
      err = encode_output(&o[i].out, g.out, g.ldout, g.P, g.Q, bf16, columns);
      if (err == cudaSuccess && g.z) err = encode_output(&o[i].z_gate, g.z, g.ldz, g.P, g.Q, bf16, columns);
      if (err == cudaSuccess && a.z_up) err = encode_output(&o[i].z_up, a.z_up, a.ldz_up, g.P, g.Q, bf16, columns);
      if (err != cudaSuccess) return err;
    }
  const auto run = [&](auto type, auto eight) {
    constexpr int D = decltype(type)::value;
    constexpr bool kE = decltype(eight)::value;
    if (!form.wide) return launch_split<D, kE>(a, m, st);
    return form.subs == 2 ? launch_wide<D, kE, 2>(a, m, o, sms, st) : launch_wide<D, kE, 1>(a, m, o, sms, st);
  };
  using Bf16 = std::integral_constant<int, ARX_BF16>;
  using F16 = std::integral_constant<int, ARX_F16>;
  if (k8) return bf16 ? run(Bf16{}, std::true_type{}) : run(F16{}, std::true_type{});
  return bf16 ? run(Bf16{}, std::false_type{}) : run(F16{}, std::false_type{});
}

}  // namespace arx
