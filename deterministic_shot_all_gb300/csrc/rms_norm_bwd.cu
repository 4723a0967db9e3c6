// Root-mean-square norm, backward: with v = dy weight and n = h rstd,
//   dx = rstd (v - n mean(v n)) + dresidual,  dweight = sum over rows of dy n.
//
// Bound by HBM: dy, h and dresidual are read and dx is written once.
// Persistent, as the layer norm's backward kernel: T threads to a row, RPC rows
// to a block, up to 16 columns to a thread (32 in the longest rows); the block's
// rows are RPC b, RPC (b + G), ... and come in through a ring of kRing rows in
// shared memory; its columns' sums of dy n stay in registers and go to the
// workspace once, as part[b][cols], for column_sum_kernel to add the blocks in
// order.  [8192, 4096] bf16 with dresidual 42.7 us, 6.3 TB/s, about 2 of it the
// column sums; [3001, 5003] in 32 bits, off 16 bytes and so element by element, 36.4
// us, 4.9 TB/s, bound by issue slots and one row's chain of sums at a time.
#include <cuda_runtime.h>

#include "arx_internal.h"
#include "norm.cuh"
#include "ops_launch.h"

namespace arx {
namespace {

constexpr unsigned kSms = 152;

template <int T, int RPC, int NV, int V>
constexpr int kBlocks = T * RPC <= 256 || (T == 512 && NV * V == 8) ? 2 : 1;

// Weights and n stay in registers, beside v; else n is worked out twice and the
// weights come from shared memory, [cols] behind the rings, if there is room, or
// from L1; and where two rows of three arrays have no room, dresidual does not come
// through the ring.  ([2432, 12288] bf16 with dresidual: 72.5 us with all of it
// from L1 and worked out twice.)
template <int T, int NV, int V>
constexpr bool kHolds = NV * V <= (T <= 512 ? 16 : 8);

template <int D, int T, int RPC, int NV, int V, int kRing>
__global__ void __launch_bounds__(T* RPC, kBlocks<T, RPC, NV, V>)
    rms_bwd_kernel(const __grid_constant__ arx_rms_norm_bwd_args a, uint32_t slot, float inv_cols, uint32_t res_ring,
                   uint32_t weights) {
  using S = typename Elem<D>::S;
  constexpr int kWarps = T / 32;
  constexpr bool kHold = kHolds<T, NV, V>;
  __shared__ float buf[2][RPC][kWarps];
  extern __shared__ __align__(16) uint8_t smem[];  // [RPC][kRing][h, dy and, with res_ring, dresidual][slot]
  dependent_launch_prologue();
  const uint32_t cols = uint32_t(a.cols);
  const bool res = a.dresidual && a.dx;
  const uint32_t arrays = res_ring ? 3 : 2, sub = threadIdx.x / T;
  uint8_t* ring = smem + sub * kRing * arrays * slot;
  const S *gh = static_cast<const S*>(a.h), *gdy = static_cast<const S*>(a.dy),
          *gdr = static_cast<const S*>(a.dresidual);

  const auto start = [&](size_t row, uint32_t at) {  // one group, empty past the last row
    if (row < a.rows) {
      uint8_t* dst = ring + at * arrays * slot;
      copy_matrix_row<D, T, NV, V>(dst, gh, a.ldh, row, a.rows, cols);
      copy_matrix_row<D, T, NV, V>(dst + slot, gdy, a.lddy, row, a.rows, cols);
      if (res_ring) copy_matrix_row<D, T, NV, V>(dst + 2 * slot, gdr, a.lddresidual, row, a.rows, cols);
    }
    cp_async_commit();
    // A dresidual that has no room in the ring is on its way to L2 at least.
    if (!kHold && res && !res_ring && row < a.rows)
      for (uint32_t c = threadIdx.x % T * (128 / sizeof(S)); c < cols; c += T * (128 / sizeof(S))) prefetch_l2_line(gdr + row * a.lddresidual + c);
  };

  float acc[NV][V] = {}, w[kHold ? NV : 1][V];
  const size_t step = size_t(gridDim.x) * RPC;
  size_t row = size_t(blockIdx.x) * RPC + sub;
#pragma unroll
  for (int i = 0; i + 1 < kRing; ++i) start(row + i * step, i);
  if constexpr (kHold) hold_params<T, NV, V>(w, a.weight, a.wdtype, cols, 1.0f);
  float* held = nullptr;  // of a block with one row at a time
  if constexpr (!kHold)
    if (weights && a.weight) {
      held = reinterpret_cast<float*>(smem + kRing * arrays * slot);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const uint32_t c = row_col<T, V>(i);
        float g[V];
        if (c < cols) {
          load_params<V>(a.weight, a.wdtype, c, g);
#pragma unroll
          for (int k = 0; k < V; ++k) held[c + k] = g[k];  // this thread's own columns: no barrier
        }
      }
    }
  float rstd = row < a.rows ? a.rstd[row] : 0.0f;
  uint32_t at = 0;
  int parity = 0;
  for (; row < a.rows; row += step) {
    const float next_rstd = row + step < a.rows ? a.rstd[row + step] : 0.0f;
    cp_async_wait<kRing - 2>();
    if (V == 1) row_barrier<T, RPC>();
    // The slot of the row before, which every thread has read for the last time.
    start(row + (kRing - 1) * step, at == 0 ? kRing - 1 : at - 1);
    const uint8_t* base = ring + at * arrays * slot;
    const uint8_t* h = base + row_offset<V>(gh + row * a.ldh);
    const uint8_t* dy = base + slot + row_offset<V>(gdy + row * a.lddy);
    const uint8_t* dr = base + 2 * slot + row_offset<V>(gdr + row * a.lddresidual);
    float n[kHold ? NV : 1][V], v[NV][V], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t c = row_col<T, V>(i);
      if (c >= cols) continue;
      float (&un)[V] = n[kHold ? i : 0], (&uv)[V] = v[i], g[V];
      read_shared<D, V>(h + c * sizeof(S), un);
      read_shared<D, V>(dy + c * sizeof(S), uv);
      if constexpr (!kHold) {
#pragma unroll
        for (int k = 0; k < V; ++k) g[k] = 1.0f;
        if (held)
          read_shared<ARX_F32, V>(reinterpret_cast<const uint8_t*>(held + c), g);
        else if (a.weight)
          load_params<V>(a.weight, a.wdtype, c, g);
      }
#pragma unroll
      for (int k = 0; k < V; ++k) {
        un[k] *= rstd;
        acc[i][k] += uv[k] * un[k];
        uv[k] *= kHold ? w[kHold ? i : 0][k] : g[k];
        sum += uv[k] * un[k];
      }
    }
    if (a.dx) {
      const float mean = row_sum<T, RPC>(sum, buf[parity][sub]) * inv_cols;
      parity ^= 1;
      S* dx = static_cast<S*>(a.dx) + row * a.lddx;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const uint32_t c = row_col<T, V>(i);
        if (c >= cols) continue;
        float (&un)[V] = n[kHold ? i : 0], o[V];
        if constexpr (!kHold) {
          read_shared<D, V>(h + c * sizeof(S), un);
#pragma unroll
          for (int k = 0; k < V; ++k) un[k] *= rstd;
        }
#pragma unroll
        for (int k = 0; k < V; ++k) o[k] = 0.0f;
        if (res_ring) {
          read_shared<D, V>(dr + c * sizeof(S), o);
        } else if (!kHold && res) {
          Pack<D, V> r;
          r.load(gdr + row * a.lddresidual + c);
          r.get(o);
        }
#pragma unroll
        for (int k = 0; k < V; ++k) o[k] += rstd * (v[i][k] - un[k] * mean);
        Pack<D, V> out;
        out.set(o);
        out.store(dx + c);
      }
    }
    rstd = next_rstd;
    at = at + 1 == kRing ? 0 : at + 1;
  }
  cp_async_wait<0>();
  if (!a.dweight) return;
  float* join = reinterpret_cast<float*>(smem);  // RPC > 1: [RPC][cols], once the rings are done with
  float* to = static_cast<float*>(a.workspace) + size_t(blockIdx.x) * cols;
  if (RPC > 1) __syncthreads();
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const uint32_t c = row_col<T, V>(i);
    float* p = (RPC > 1 ? join + sub * cols : to) + c;
    if (c >= cols) continue;
    if constexpr (V == 8) {
      reinterpret_cast<float4*>(p)[0] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
    } else {
      p[0] = acc[i][0];
    }
  }
  if constexpr (RPC > 1) {
    __syncthreads();
    for (uint32_t c = threadIdx.x; c < cols; c += T * RPC) {
      float s = join[c];
#pragma unroll
      for (int r = 1; r < RPC; ++r) s += join[r * cols + c];
      to[c] = s;
    }
  }
}

// Any row length: dx with two passes over the row, and the column sums by
// rms_bwd_columns_kernel.
template <int D>
__global__ void __launch_bounds__(512) rms_bwd_long_kernel(const __grid_constant__ arx_rms_norm_bwd_args a) {
  using S = typename Elem<D>::S;
  __shared__ float buf[16];
  dependent_launch_prologue();
  const size_t row = blockIdx.x;
  const S* h = static_cast<const S*>(a.h) + row * a.ldh;
  const S* dy = static_cast<const S*>(a.dy) + row * a.lddy;
  const S* dr = a.dresidual ? static_cast<const S*>(a.dresidual) + row * a.lddresidual : nullptr;
  S* dx = static_cast<S*>(a.dx) + row * a.lddx;
  const float rstd = a.rstd[row];
  float s = 0.0f;
  for (size_t c = threadIdx.x; c < a.cols; c += 512) {
    float v = Elem<D>::widen(dy[c]);
    if (a.weight) v *= load_param(a.weight, a.wdtype, c);
    s += v * (Elem<D>::widen(h[c]) * rstd);
  }
  const float mean = row_sum<512, 1>(s, buf) / float(a.cols);
  for (size_t c = threadIdx.x; c < a.cols; c += 512) {
    float v = Elem<D>::widen(dy[c]);
    if (a.weight) v *= load_param(a.weight, a.wdtype, c);
    const float o = rstd * (v - Elem<D>::widen(h[c]) * rstd * mean);
    dx[c] = Elem<D>::round(dr ? o + Elem<D>::widen(dr[c]) : o);
  }
}

// part[blockIdx.y][col] over the rows of chunk blockIdx.y.
template <int D>
__global__ void __launch_bounds__(256) rms_bwd_columns_kernel(const __grid_constant__ arx_rms_norm_bwd_args a) {
  using S = typename Elem<D>::S;
  __shared__ float join[8][32];
  dependent_launch_prologue();
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const size_t c = size_t(blockIdx.x) * 32 + tx;
  float s = 0.0f;
  if (c < a.cols)
    for (size_t row = size_t(blockIdx.y) * 8 + ty; row < a.rows; row += size_t(gridDim.y) * 8)
      s += Elem<D>::widen(static_cast<const S*>(a.dy)[row * a.lddy + c]) *
           (Elem<D>::widen(static_cast<const S*>(a.h)[row * a.ldh + c]) * a.rstd[row]);
  join[ty][tx] = s;
  __syncthreads();
  if (ty == 0 && c < a.cols) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += join[i][tx];
    static_cast<float*>(a.workspace)[size_t(blockIdx.y) * a.cols + c] = s;
  }
}

// Shared memory of an SM that its blocks' rings may fill, and of one block.
constexpr size_t kRingBytes = 222 * 1024, kBlockRingBytes = 220 * 1024;
// Row chunks of the column-sum kernel for long rows.
constexpr unsigned kColumnChunks = 64;

// As many blocks as 152 SMs hold at once: a constant, so that the order of the
// sums depends on the call alone: sizes, type, alignment, and whether dresidual (an
// array more in the ring) is there.
template <int D, int T, int RPC, int NV, int V, int kRing>
cudaError_t ring(const arx_rms_norm_bwd_args& a, unsigned* parts, uint32_t slot, bool res_ring, cudaStream_t st) {
  size_t smem = size_t(kRing) * (res_ring ? 3 : 2) * slot * RPC;
  const size_t params = RPC == 1 && a.weight ? a.cols * 4 : 0;
  const bool weights = params && smem + params <= kBlockRingBytes && !kHolds<T, NV, V>;
  if (weights) smem += params;
  size_t per_sm = kRingBytes / (smem + 2048);
  if (per_sm > kBlocks<T, RPC, NV, V>) per_sm = kBlocks<T, RPC, NV, V>;
  if (per_sm < 1) per_sm = 1;
  const uint64_t need = (a.rows + RPC - 1) / RPC;
  const unsigned blocks = unsigned(need < per_sm * kSms ? need : per_sm * kSms);
  *parts = blocks;
  constexpr auto kernel = rms_bwd_kernel<D, T, RPC, NV, V, kRing>;
  const cudaError_t e = allow_dynamic_smem<kernel>(kBlockRingBytes);
  if (e != cudaSuccess) return e;
  return launch_op(kernel, dim3(blocks), T * RPC, smem, st, a, slot, 1.0f / float(a.cols), uint32_t(res_ring),
                   uint32_t(weights));
}

// Three rows in the ring, two where three are too large, of the longest rows
// without dresidual; *done is false where two are too large as well.
template <int D, int T, int RPC, int NV, int V>
cudaError_t run(const arx_rms_norm_bwd_args& a, unsigned* parts, bool* done, cudaStream_t st) {
  const uint32_t slot = row_slot(a.cols, sizeof(typename Elem<D>::S), V);
  const bool res = a.dresidual && a.dx;
  const size_t row = size_t(res ? 3 : 2) * slot * RPC;
  *done = true;
  // (Two rows of two arrays hold the RPC rows of sums, too.)
  if (3 * row <= kBlockRingBytes) return ring<D, T, RPC, NV, V, 3>(a, parts, slot, res, st);
  if (2 * row <= kBlockRingBytes) return ring<D, T, RPC, NV, V, 2>(a, parts, slot, res, st);
  if constexpr (!kHolds<T, NV, V>)
    if (size_t(4) * slot <= kBlockRingBytes) return ring<D, T, RPC, NV, V, 2>(a, parts, slot, false, st);
  *done = false;
  return cudaSuccess;
}

// 512 threads to 16-bit rows of 2049 to 4096 columns, whose rings leave room for two
// blocks on an SM ([8192, 4096] with dresidual: 46.0 us against 47.0 with 256 threads;
// with 256 and two rows in the ring of three blocks 54.6); 640 to rows of 4097 to
// 5120 columns off 16 bytes ([3001, 5003] in 32 bits: 36.0 against 37.4 with 320).
template <int D>
cudaError_t any(const arx_rms_norm_bwd_args& a, bool vec, unsigned* parts, cudaStream_t st) {
  const uint64_t n = a.cols;
  bool done = true;
  cudaError_t e = cudaSuccess;
  if (vec) {
    if (n <= 256)
      e = run<D, 32, 8, 1, 8>(a, parts, &done, st);
    else if (n <= 512)
      e = run<D, 32, 8, 2, 8>(a, parts, &done, st);
    else if (n <= 1024)
      e = run<D, 64, 4, 2, 8>(a, parts, &done, st);
    else if (n <= 2048)
      e = run<D, 128, 2, 2, 8>(a, parts, &done, st);
    else if (n <= 4096 && D != ARX_F32)
      e = run<D, 512, 1, 1, 8>(a, parts, &done, st);
    else if (n <= 4096)
      e = run<D, 256, 1, 2, 8>(a, parts, &done, st);
    else if (n <= 8192)
      e = run<D, 512, 1, 2, 8>(a, parts, &done, st);
    else if (n <= 16384)
      e = run<D, 512, 1, 4, 8>(a, parts, &done, st);
    else
      done = false;
  } else {
    if (n <= 256)
      e = run<D, 32, 8, 8, 1>(a, parts, &done, st);
    else if (n <= 512)
      e = run<D, 32, 8, 16, 1>(a, parts, &done, st);
    else if (n <= 1024)
      e = run<D, 64, 4, 16, 1>(a, parts, &done, st);
    else if (n <= 2048)
      e = run<D, 128, 2, 16, 1>(a, parts, &done, st);
    else if (n <= 4096)
      e = run<D, 256, 1, 16, 1>(a, parts, &done, st);
    else if (n <= 5120)
      e = run<D, 640, 1, 8, 1>(a, parts, &done, st);
    else if (n <= 8192)
      e = run<D, 512, 1, 16, 1>(a, parts, &done, st);
    else if (n <= 16384)
      e = run<D, 1024, 1, 16, 1>(a, parts, &done, st);
    else
      done = false;
  }
  if (e != cudaSuccess || done) return e;
  // The column sums first: dx may be written over dy or h.
  *parts = 0;
  if (a.dweight) {
    const uint64_t need = (a.rows + 7) / 8;
    *parts = unsigned(need < kColumnChunks ? need : kColumnChunks);
    const dim3 grid(unsigned((a.cols + 31) / 32), *parts);
    const cudaError_t c = launch_op(rms_bwd_columns_kernel<D>, grid, 256, 0, st, a);
    if (c != cudaSuccess) return c;
  }
  if (!a.dx) return cudaSuccess;
  return launch_op(rms_bwd_long_kernel<D>, dim3(unsigned(a.rows)), 512, 0, st, a);
}

}  // namespace

// An upper bound: kBlocks to an SM, or the chunks of the long form.
size_t rms_bwd_parts(uint64_t rows) { return size_t(rows < 2 * kSms ? rows : 2 * kSms); }

cudaError_t launch_rms_norm_bwd(const arx_rms_norm_bwd_args& a, bool vec, cudaStream_t st) {
  unsigned parts = 0;
  if (a.rows > 0) {
    const cudaError_t e = a.dtype == ARX_BF16  ? any<ARX_BF16>(a, vec, &parts, st)
                          : a.dtype == ARX_F16 ? any<ARX_F16>(a, vec, &parts, st)
                                               : any<ARX_F32>(a, vec, &parts, st);
    if (e != cudaSuccess) return e;
  }
  return launch_column_sum(static_cast<const float*>(a.workspace), parts, a.cols, a.dweight, nullptr, nullptr,
                           a.wdtype, st);
}

}  // namespace arx
