// The gradients of a gated block's projections, the first step of its backward
// pass: dg = dout u act'(g), du = dout act(g), and the sums of their columns.
//
// Bound by HBM, elementwise: three matrices are read and two written once
// (tiles.cuh has the tiles and the sums).  dg and du are rounded to the
// operands' type where they are stored, as the tensor cores take no other
// beside 16-bit weights and activations; the column sums take them unrounded.
// act and act' share their exponential and quotient, and a thread has one row's
// three units in flight, so that three blocks fit an SM with registers to spare:
// [8185, 4096] with silu 8 us less than with two rows and both functions worked
// out apart (57.5), three rows 24 us more.
#include <cuda_runtime.h>

#include "activation.cuh"
#include "arx_internal.h"
#include "tiles.cuh"

namespace arx {
namespace {

template <int D, int kAccess>
__global__ void __launch_bounds__(kTileThreads, kTileBlocks) gated_grad_kernel(const GatedGradCall a, Tile t) {
  using G = Group<D, kAccess>;
  using S = typename Elem<D>::S;
  __shared__ __align__(16) uint8_t stages[kTileThreads / 32 * G::kStageBytes + 16];
  S* stage = reinterpret_cast<S*>(stages + threadIdx.x / 32 * G::kStageBytes);
  dependent_launch_prologue();
  const Columns<D, kAccess> c(t, a.cols);
  float sum_g[8] = {}, sum_u[8] = {};
  if (c.any) {
    const S* dout = static_cast<const S*>(a.dout) + c.at;
    const S* zg = static_cast<const S*>(a.z_gate) + c.at;
    const S* zu = static_cast<const S*>(a.z_up) + c.at;
    S* dz = static_cast<S*>(a.dz) + c.at;
    const size_t step = size_t(gridDim.y) * t.rows();
    for (size_t row = size_t(blockIdx.y) * t.rows() + t.ty(); row < a.rows; row += step) {
      G vd, vg, vu;
      vd.load(dout + row * a.lddout, c.n);
      vg.load(zg + row * a.ldz_gate, c.n);
      vu.load(zu + row * a.ldz_up, c.n);
      float d[8], g[8], dg[8];
      vd.get(d, stage);
      vu.get(dg, stage);
      vg.get(g, stage);
#pragma unroll
      for (int k = 0; k < 8; ++k) dg[k] *= d[k];
      multiply_activation_both<8>(dg, d, g, a.act);
#pragma unroll
      for (int k = 0; k < 8; ++k) sum_g[k] += dg[k], sum_u[k] += d[k];
      if (a.dz) {
        G::put(dz + row * a.lddz, dg, c.n, stage);
        G::put(dz + row * a.lddz + a.du, d, c.n, stage);
      }
    }
  }
  if (a.dbias_gate) store_part(sum_g, t, c.first, a.cols, a.part);
  if (a.dbias_up) {
    __syncthreads();
    store_part(sum_u, t, c.first, a.cols, a.part + size_t(gridDim.y) * a.cols);
  }
}

template <int D>
cudaError_t gated_grad(const GatedGradCall& c, bool vec, cudaStream_t st) {
  return with_access(vec, c.cols, [&](auto m) {
    return launch_op(gated_grad_kernel<D, decltype(m)::value>, tile_grid(c.rows, c.cols), kTileThreads, 0, st, c,
                     tile_of(c.cols));
  });
}

}  // namespace

cudaError_t launch_gated_grad(const GatedGradCall& c, bool vec, cudaStream_t st) {
  unsigned parts = 0;
  if (c.rows > 0) {
    parts = row_chunks(c.rows, c.cols);
    const cudaError_t e = c.dtype == ARX_BF16 ? gated_grad<ARX_BF16>(c, vec, st) : gated_grad<ARX_F16>(c, vec, st);
    if (e != cudaSuccess) return e;
  }
  return launch_column_sum(c.part, parts, c.cols, c.dbias_gate, c.part + size_t(parts) * c.cols, c.dbias_up, c.wdtype, st);
}

}  // namespace arx
