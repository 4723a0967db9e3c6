// The end of a sublayer in one kernel: rank-order sum of W bf16 partials, residual,
// root-mean-square norm (rms_norm.cuh has the kernels).
#include "rms_norm.cuh"

namespace arx {

cudaError_t launch_reduce_rms_norm(const arx_reduce_rms_norm_args& c, bool vec, cudaStream_t st) {
  RmsArgs<ARX_BF16> a{};
  for (int r = 0; r < c.W; ++r) a.slot[r] = static_cast<const uint16_t*>(c.slots[r]);
  a.residual = static_cast<const uint16_t*>(c.residual);
  a.weight = c.weight, a.wdtype = ARX_BF16, a.W = c.W;
  a.h = static_cast<uint16_t*>(c.h), a.y = static_cast<uint16_t*>(c.y);
  a.q = static_cast<uint8_t*>(c.q), a.scale = c.scale, a.rstd = c.rstd;
  a.rows = c.rows, a.cols = c.cols;
  a.ldx = a.ldresidual = a.ldh = a.ldy = c.cols, a.ldq = c.ldq;
  a.eps = c.eps, a.inv_cols = 1.0f / float(c.cols);
  const auto place = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16; };
  a.alike = place(c.weight) == 0;
  for (const void* p : {c.residual, static_cast<const void*>(c.h), static_cast<const void*>(c.y)})
    a.alike = a.alike && (!p || place(p) == place(c.slots[0]));
  for (int r = 1; r < c.W; ++r) a.alike = a.alike && place(c.slots[r]) == place(c.slots[0]);
  switch (c.W) {
    case 1: return run_w<ARX_BF16, 1>(a, vec, st);
    case 2: return run_w<ARX_BF16, 2>(a, vec, st);
    case 3: return run_w<ARX_BF16, 3>(a, vec, st);
    case 4: return run_w<ARX_BF16, 4>(a, vec, st);
    case 5: return run_w<ARX_BF16, 5>(a, vec, st);
    case 6: return run_w<ARX_BF16, 6>(a, vec, st);
    case 7: return run_w<ARX_BF16, 7>(a, vec, st);
    case 8: return run_w<ARX_BF16, 8>(a, vec, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace arx
