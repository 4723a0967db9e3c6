// Root-mean-square norm with the residual's addition (rms_norm.cuh has the kernels).
#include "rms_norm.cuh"

namespace arx {
namespace {

template <int D>
cudaError_t rms_norm(const arx_rms_norm_args& c, bool vec, cudaStream_t st) {
  using S = typename Elem<D>::S;
  RmsArgs<D> a{};
  a.slot[0] = static_cast<const S*>(c.x);
  a.residual = static_cast<const S*>(c.residual);
  a.weight = c.weight, a.wdtype = c.wdtype, a.W = 1;
  a.h = static_cast<S*>(c.h), a.y = static_cast<S*>(c.y);
  a.q = static_cast<uint8_t*>(c.q), a.scale = c.scale, a.rstd = c.rstd;
  a.rows = c.rows, a.cols = c.cols;
  a.ldx = c.ldx, a.ldresidual = c.ldresidual, a.ldh = c.ldh, a.ldy = c.ldy, a.ldq = c.ldq;
  a.eps = c.eps, a.inv_cols = 1.0f / float(c.cols);
  // Contiguous matrices that begin alike.
  const auto alike = [&](const void* p, uint64_t ld) {
    return !p || (reinterpret_cast<uintptr_t>(p) % 16 == reinterpret_cast<uintptr_t>(c.x) % 16 && (c.rows <= 1 || ld == c.cols));
  };
  a.alike = c.wdtype == c.dtype && reinterpret_cast<uintptr_t>(c.weight) % 16 == 0 && alike(c.x, c.ldx) &&
            alike(c.residual, c.ldresidual) && alike(c.h, c.ldh) && alike(c.y, c.ldy);
  return run_w<D, 1>(a, vec, st);
}

}  // namespace

cudaError_t launch_rms_norm(const arx_rms_norm_args& c, bool vec, cudaStream_t st) {
  if (c.dtype == ARX_BF16) return rms_norm<ARX_BF16>(c, vec, st);
  if (c.dtype == ARX_F16) return rms_norm<ARX_F16>(c, vec, st);
  return rms_norm<ARX_F32>(c, vec, st);
}

}  // namespace arx
