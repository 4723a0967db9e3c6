// C entry points of the operators of a sublayer with a root-mean-square norm
// and a gated feed-forward block: argument checks on the host, then the
// launchers.
#include <cuda_runtime.h>

#include <cstdint>

#include "arx.h"
#include "arx_internal.h"
#include "ops_check.h"
#include "ops_launch.h"

namespace {

using namespace arx::ops;
using arx::report;

}  // namespace

extern "C" {

arx_status arx_rms_norm(const arx_rms_norm_args* a, void* stream) {
  if (!a) return report(ARX_EINVAL, "null arguments");
  ARX_TRY(check_types(a->dtype, a->wdtype, true));
  ARX_TRY(check_dims(a->rows, a->cols, 0));
  ARX_TRY(check_eps(a->eps));
  if (a->rows == 0 || a->cols == 0) return ok();
  if (!a->y && !a->q) return report(ARX_EINVAL, "y and q are null");
  const Mat in[] = {mat("x", a->x, a->rows, a->cols, a->ldx, a->dtype),
                    mat("residual", a->residual, a->rows, a->cols, a->ldresidual, a->dtype),
                    vec("weight", a->weight, a->cols, a->wdtype)};
  const Mat out[] = {mat("h", a->h, a->rows, a->cols, a->ldh, a->dtype),
                     mat("y", a->y, a->rows, a->cols, a->ldy, a->dtype),
                     mat("q", a->q, a->rows, a->cols, a->ldq, ARX_E4M3),
                     vec("scale", a->q ? a->scale : nullptr, a->rows, ARX_F32), vec("rstd", a->rstd, a->rows, ARX_F32)};
  for (int i = 0; i < 3; ++i) ARX_TRY(check_mat(in[i], i == 0));
  for (int i = 0; i < 5; ++i) {
    ARX_TRY(check_mat(out[i], i == 3 && a->q));
    ARX_TRY(check_output(out[i], in, 3, i < 2 ? 3u : 0u));
    ARX_TRY(check_output(out[i], out, i, 0));
  }
  const bool v = units(in[0]) && units(in[1]) && units(out[0]) && units(out[1]) && units(out[2]) && param_units(a->weight);
  return launched(arx::launch_rms_norm(*a, v, static_cast<cudaStream_t>(stream)), "arx_rms_norm");
}

size_t arx_rms_norm_bwd_workspace_bytes(uint64_t rows, uint64_t cols) {
  if (rows > kMaxDim || cols > kMaxDim) return 0;
  return size_t(arx::rms_bwd_parts(rows) * cols * 4);
}

arx_status arx_rms_norm_bwd(const arx_rms_norm_bwd_args* a, void* stream) {
  if (!a) return report(ARX_EINVAL, "null arguments");
  ARX_TRY(check_types(a->dtype, a->wdtype, true));
  ARX_TRY(check_dims(a->rows, a->cols, 0));
  if (a->cols == 0 || (!a->dx && !a->dweight)) return ok();
  const Mat in[] = {mat("dy", a->dy, a->rows, a->cols, a->lddy, a->dtype),
                    mat("h", a->h, a->rows, a->cols, a->ldh, a->dtype),
                    mat("dresidual", a->dresidual, a->rows, a->cols, a->lddresidual, a->dtype),
                    vec("rstd", a->rstd, a->rows, ARX_F32), vec("weight", a->weight, a->cols, a->wdtype)};
  const uint64_t need = a->dweight ? arx_rms_norm_bwd_workspace_bytes(a->rows, a->cols) : 0;
  const Mat out[] = {mat("dx", a->dx, a->rows, a->cols, a->lddx, a->dtype), vec("dweight", a->dweight, a->cols, a->wdtype),
                     vec("workspace", need ? a->workspace : nullptr, need / 4, ARX_F32)};
  ARX_TRY(check_workspace(a->workspace, a->workspace_bytes, need));
  for (int i = 0; i < 5; ++i) ARX_TRY(check_mat(in[i], i != 2 && i != 4));
  for (int i = 0; i < 3; ++i) {
    ARX_TRY(check_mat(out[i], false));
    ARX_TRY(check_output(out[i], in, 5, i == 0 ? 7u : 0u));
    ARX_TRY(check_output(out[i], out, i, 0));
  }
  const bool v = units(in[0]) && units(in[1]) && units(in[2]) && units(out[0]) && param_units(a->weight);
  return launched(arx::launch_rms_norm_bwd(*a, v, static_cast<cudaStream_t>(stream)), "arx_rms_norm_bwd");
}

arx_status arx_reduce_rms_norm(const arx_reduce_rms_norm_args* a, void* stream) {
  if (!a) return report(ARX_EINVAL, "null arguments");
  if (a->W < 1 || a->W > ARX_MAX_W) return report(ARX_EINVAL, "W=%d outside 1..%d", a->W, ARX_MAX_W);
  ARX_TRY(check_dims(a->rows, a->cols, 0));
  ARX_TRY(check_eps(a->eps));
  if (a->rows == 0 || a->cols == 0) return ok();
  if (!a->slots) return report(ARX_EINVAL, "null pointer array");
  if (!a->y && !a->q) return report(ARX_EINVAL, "y and q are null");
  Mat in[ARX_MAX_W + 2];
  int n = 0;
  in[n++] = mat("residual", a->residual, a->rows, a->cols, a->cols, ARX_BF16);
  for (int r = 0; r < a->W; ++r) in[n++] = mat("a slot", a->slots[r], a->rows, a->cols, a->cols, ARX_BF16);
  const int matrices = n;
  in[n++] = vec("weight", a->weight, a->cols, ARX_BF16);
  const Mat out[] = {mat("h", a->h, a->rows, a->cols, a->cols, ARX_BF16),
                     mat("y", a->y, a->rows, a->cols, a->cols, ARX_BF16),
                     mat("q", a->q, a->rows, a->cols, a->ldq, ARX_E4M3),
                     vec("scale", a->q ? a->scale : nullptr, a->rows, ARX_F32), vec("rstd", a->rstd, a->rows, ARX_F32)};
  for (int i = 0; i < n; ++i) ARX_TRY(check_mat(in[i], i >= 1 && i < matrices));
  for (int i = 0; i < 5; ++i) {
    ARX_TRY(check_mat(out[i], i == 3 && a->q));
    ARX_TRY(check_output(out[i], in, n, i < 2 ? (1u << matrices) - 1u : 0u));
    ARX_TRY(check_output(out[i], out, i, 0));
  }
  bool v = units(out[0]) && units(out[1]) && units(out[2]) && param_units(a->weight);
  for (int i = 0; i < matrices; ++i) v = v && units(in[i]);
  return launched(arx::launch_reduce_rms_norm(*a, v, static_cast<cudaStream_t>(stream)), "arx_reduce_rms_norm");
}

}  // extern "C"
