// C entry points of the operators around the reduce: argument checks on the
// host, then the launchers.
#include <cuda_runtime.h>

#include <cstdint>

#include "arx.h"
#include "arx_internal.h"
#include "ops_check.h"
#include "ops_launch.h"

namespace {

using namespace arx::ops;
using arx::report;

arx::GemmCall forward_product(const arx_linear_args& a) {
  return product(a.x, a.ldx, false, a.w, a.ldw, false, a.M, a.N, a.K, a.dtype, a.wdtype, a.status,
                 a.wait_us);
}
// dx = dz w: w's rows are the contraction.
arx::GemmCall dx_product(const arx_linear_bwd_args& a, const void* dz, uint64_t lddz) {
  return product(dz, lddz, false, a.w, a.ldw, true, a.M, a.K, a.N, a.dtype, a.wdtype, a.status,
                 a.wait_us);
}
// dw = dz^T x: the rows of both are.
arx::GemmCall dw_product(const arx_linear_bwd_args& a, const void* dz, uint64_t lddz) {
  return product(dz, lddz, true, a.x, a.ldx, true, a.N, a.K, a.M, a.dtype, a.wdtype, a.status,
                 a.wait_us);
}

// Where the products of a backward pass find dz: in the workspace (rows of N
// rounded up to 8), or dout itself without an activation -- unless its rows are
// off 16 bytes and there is a workspace: a copy on aligned rows costs its
// bytes, and both products load their larger operand by the copy engine
// ([1001, 2047] x 2049: 148 us without, 117 with).
bool dz_in_workspace(const arx_linear_bwd_args& a) {
  if (!a.dx && !a.dw) return false;
  if (a.act != ARX_ACT_NONE) return true;
  const bool off = reinterpret_cast<uintptr_t>(a.dout) % 16 || (a.M > 1 && a.lddout % 8);
  return off && a.workspace && reinterpret_cast<uintptr_t>(a.workspace) % 16 == 0 &&
         a.workspace_bytes >= arx_linear_bwd_workspace_bytes(a.M, a.N);
}

size_t backward_copies_bytes(const arx_linear_bwd_args& a) {
  const bool ws = dz_in_workspace(a);
  // Any address on 16 bytes stands for a workspace that is not there yet.
  const void* dz = ws ? reinterpret_cast<const void*>(uintptr_t(16)) : a.dout;
  const uint64_t lddz = ws ? (a.N + 7) / 8 * 8 : a.lddout;
  const size_t dx = a.dx ? arx::gemm_copies_bytes(dx_product(a, dz, lddz)) : 0,
               dw = a.dw ? arx::gemm_copies_bytes(dw_product(a, dz, lddz)) : 0;
  return dx > dw ? dx : dw;
}

}  // namespace

extern "C" {

arx_status arx_layer_norm(const arx_layer_norm_args* a, void* stream) {
  if (!a) return report(ARX_EINVAL, "null arguments");
  ARX_TRY(check_types(a->dtype, a->wdtype, true));
  ARX_TRY(check_dims(a->rows, a->cols, 0));
  ARX_TRY(check_eps(a->eps));
  if (a->rows == 0 || a->cols == 0) return ok();
  const Mat in[] = {mat("x", a->x, a->rows, a->cols, a->ldx, a->dtype), vec("weight", a->weight, a->cols, a->wdtype),
                    vec("bias", a->bias, a->cols, a->wdtype)};
  const Mat out[] = {mat("y", a->y, a->rows, a->cols, a->ldy, a->dtype), vec("mean", a->mean, a->rows, ARX_F32),
                     vec("rstd", a->rstd, a->rows, ARX_F32)};
  for (int i = 0; i < 3; ++i) ARX_TRY(check_mat(in[i], i == 0));
  for (int i = 0; i < 3; ++i) ARX_TRY(check_mat(out[i], i == 0));
  for (int i = 0; i < 3; ++i) {
    ARX_TRY(check_output(out[i], in, 3, i == 0 ? 1u : 0u));
    ARX_TRY(check_output(out[i], out, i, 0));
  }
  const bool v = units(in[0]) && units(out[0]) && param_units(a->weight) && param_units(a->bias);
  return launched(arx::launch_layer_norm(*a, v, static_cast<cudaStream_t>(stream)), "arx_layer_norm");
}

size_t arx_layer_norm_bwd_workspace_bytes(uint64_t rows, uint64_t cols) {
  if (rows > kMaxDim || cols > kMaxDim) return 0;
  return size_t(2 * arx::norm_bwd_parts(rows, cols) * cols * 4);
}

arx_status arx_layer_norm_bwd(const arx_layer_norm_bwd_args* a, void* stream) {
  if (!a) return report(ARX_EINVAL, "null arguments");
  ARX_TRY(check_types(a->dtype, a->wdtype, true));
  ARX_TRY(check_dims(a->rows, a->cols, 0));
  if (a->cols == 0 || (!a->dx && !a->dweight && !a->dbias)) return ok();
  const Mat in[] = {mat("dy", a->dy, a->rows, a->cols, a->lddy, a->dtype),
                    mat("x", a->x, a->rows, a->cols, a->ldx, a->dtype),
                    mat("dresidual", a->dresidual, a->rows, a->cols, a->lddresidual, a->dtype),
                    vec("mean", a->mean, a->rows, ARX_F32),
                    vec("rstd", a->rstd, a->rows, ARX_F32),
                    vec("weight", a->weight, a->cols, a->wdtype)};
  const uint64_t need = a->dweight || a->dbias ? arx_layer_norm_bwd_workspace_bytes(a->rows, a->cols) : 0;
  const Mat out[] = {mat("dx", a->dx, a->rows, a->cols, a->lddx, a->dtype),
                     vec("dweight", a->dweight, a->cols, a->wdtype), vec("dbias", a->dbias, a->cols, a->wdtype),
                     vec("workspace", need ? a->workspace : nullptr, need / 4, ARX_F32)};
  ARX_TRY(check_workspace(a->workspace, a->workspace_bytes, need));
  for (int i = 0; i < 6; ++i) ARX_TRY(check_mat(in[i], i != 2 && i != 5));
  for (int i = 0; i < 4; ++i) {
    ARX_TRY(check_mat(out[i], false));
    ARX_TRY(check_output(out[i], in, 6, i == 0 ? 7u : 0u));
    ARX_TRY(check_output(out[i], out, i, 0));
  }
  const bool v = units(in[0]) && units(in[1]) && units(in[2]) && units(out[0]) && param_units(a->weight);
  return launched(arx::launch_layer_norm_bwd(*a, v, static_cast<cudaStream_t>(stream)), "arx_layer_norm_bwd");
}

arx_status arx_dropout_add(const arx_dropout_add_args* a, void* stream) {
  if (!a) return report(ARX_EINVAL, "null arguments");
  ARX_TRY(check_types(a->dtype, a->wdtype, true));
  ARX_TRY(check_dims(a->rows, a->cols, 0));
  ARX_TRY(check_dropout(a->p, a->rng));
  if (a->rows == 0 || a->cols == 0) return ok();
  const Mat in[] = {mat("x", a->x, a->rows, a->cols, a->ldx, a->dtype),
                    mat("residual", a->residual, a->rows, a->cols, a->ldresidual, a->dtype),
                    vec("bias", a->bias, a->cols, a->wdtype), vec("rng", a->rng, 4, ARX_F32)};
  const Mat out = mat("out", a->out, a->rows, a->cols, a->ldout, a->dtype);
  for (int i = 0; i < 3; ++i) ARX_TRY(check_mat(in[i], i == 0));
  ARX_TRY(check_mat(out, true));
  ARX_TRY(check_output(out, in, 4, 3u));
  const bool v = units(in[0]) && units(in[1]) && units(out);
  return launched(arx::launch_dropout_add(*a, v, static_cast<cudaStream_t>(stream)), "arx_dropout_add");
}

size_t arx_dropout_add_bwd_workspace_bytes(uint64_t rows, uint64_t cols) {
  if (rows > kMaxDim || cols > kMaxDim) return 0;
  return size_t(arx::column_parts(rows, cols) * cols * 4);
}

arx_status arx_dropout_add_bwd(const arx_dropout_add_bwd_args* a, void* stream) {
  if (!a) return report(ARX_EINVAL, "null arguments");
  ARX_TRY(check_types(a->dtype, a->wdtype, true));
  ARX_TRY(check_dims(a->rows, a->cols, 0));
  ARX_TRY(check_dropout(a->p, a->rng));
  if (a->cols == 0 || (!a->dx && !a->dbias)) return ok();
  const Mat in[] = {mat("dout", a->dout, a->rows, a->cols, a->lddout, a->dtype), vec("rng", a->rng, 4, ARX_F32)};
  const uint64_t need = a->dbias ? arx_dropout_add_bwd_workspace_bytes(a->rows, a->cols) : 0;
  const Mat out[] = {mat("dx", a->dx, a->rows, a->cols, a->lddx, a->dtype), vec("dbias", a->dbias, a->cols, a->wdtype),
                     vec("workspace", need ? a->workspace : nullptr, need / 4, ARX_F32)};
  ARX_TRY(check_workspace(a->workspace, a->workspace_bytes, need));
  ARX_TRY(check_mat(in[0], true));
  for (int i = 0; i < 3; ++i) {
    ARX_TRY(check_mat(out[i], false));
    ARX_TRY(check_output(out[i], in, 2, i == 0 ? 1u : 0u));
    ARX_TRY(check_output(out[i], out, i, 0));
  }
  const bool v = units(in[0]) && units(out[0]);
  return launched(arx::launch_dropout_add_bwd(*a, v, static_cast<cudaStream_t>(stream)), "arx_dropout_add_bwd");
}

arx_status arx_reduce_layer_norm(const arx_reduce_layer_norm_args* a, void* stream) {
  if (!a) return report(ARX_EINVAL, "null arguments");
  if (a->W < 1 || a->W > ARX_MAX_W) return report(ARX_EINVAL, "W=%d outside 1..%d", a->W, ARX_MAX_W);
  ARX_TRY(check_dims(a->rows, a->cols, 0));
  ARX_TRY(check_eps(a->eps));
  ARX_TRY(check_dropout(a->p, a->rng));
  if (a->rows == 0 || a->cols == 0) return ok();
  if (!a->slots) return report(ARX_EINVAL, "null pointer array");
  Mat in[ARX_MAX_W + 5];
  int n = 0;
  in[n++] = mat("residual", a->residual, a->rows, a->cols, a->cols, ARX_BF16);
  for (int r = 0; r < a->W; ++r) in[n++] = mat("a slot", a->slots[r], a->rows, a->cols, a->cols, ARX_BF16);
  const int matrices = n;
  in[n++] = vec("bias", a->bias, a->cols, ARX_BF16);
  in[n++] = vec("weight", a->weight, a->cols, ARX_BF16);
  in[n++] = vec("norm_bias", a->norm_bias, a->cols, ARX_BF16);
  in[n++] = vec("rng", a->rng, 4, ARX_F32);
  const Mat out[] = {mat("y", a->y, a->rows, a->cols, a->cols, ARX_BF16),
                     mat("h", a->h, a->rows, a->cols, a->cols, ARX_BF16), vec("mean", a->mean, a->rows, ARX_F32),
                     vec("rstd", a->rstd, a->rows, ARX_F32)};
  for (int i = 0; i < n; ++i) ARX_TRY(check_mat(in[i], i >= 1 && i < matrices));
  for (int i = 0; i < 4; ++i) {
    ARX_TRY(check_mat(out[i], i == 0));
    ARX_TRY(check_output(out[i], in, n, i < 2 ? (1u << matrices) - 1u : 0u));
    ARX_TRY(check_output(out[i], out, i, 0));
  }
  bool v = units(out[0]) && units(out[1]);
  for (int i = 0; i < matrices; ++i) v = v && units(in[i]);
  for (int i = matrices; i < matrices + 3; ++i) v = v && param_units(in[i].p);
  return launched(arx::launch_reduce_layer_norm(*a, v, static_cast<cudaStream_t>(stream)), "arx_reduce_layer_norm");
}

int arx_stream_capturing(void* stream) {
  cudaStreamCaptureStatus s = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(static_cast<cudaStream_t>(stream), &s) != cudaSuccess) {
    (void)cudaGetLastError();  // the default stream beside a capture that waits for it, or no device
    return 0;
  }
  return s != cudaStreamCaptureStatusNone;
}

size_t arx_linear_copies_bytes(const arx_linear_args* a) {
  if (!a || a->M > kMaxDim || a->N > kMaxDim || a->K > kMaxDim) return 0;
  return arx::gemm_copies_bytes(forward_product(*a));
}

arx_status arx_linear(const arx_linear_args* a, void* stream) {
  if (!a) return report(ARX_EINVAL, "null arguments");
  ARX_TRY(check_types(a->dtype, a->wdtype, false));
  ARX_TRY(check_dims(a->M, a->N, a->K));
  if (a->act < ARX_ACT_NONE || a->act > ARX_ACT_SILU) return report(ARX_EINVAL, "unknown activation %d", a->act);
  ARX_TRY(check_wait(a->wait_us));
  if (a->M == 0 || a->N == 0) return ok();
  arx::GemmCall c = forward_product(*a);
  const size_t copies = a->copies ? arx::gemm_copies_bytes(c) : 0;
  ARX_TRY(check_copies(a->copies, a->copies_bytes, copies));
  const Mat in[] = {mat("residual", a->residual, a->M, a->N, a->ldresidual, a->dtype),
                    mat("x", a->x, a->M, a->K, a->ldx, a->dtype), mat("w", a->w, a->N, a->K, a->ldw, a->dtype),
                    vec("bias", a->bias, a->N, a->wdtype)};
  const Mat out[] = {mat("out", a->out, a->M, a->N, a->ldout, a->dtype), mat("z", a->z, a->M, a->N, a->ldz, a->dtype),
                     vec("status", a->status, 1, ARX_F32), vec("copies", a->copies, copies / 2, ARX_BF16)};
  for (int i = 0; i < 4; ++i) ARX_TRY(check_mat(in[i], i == 1 || i == 2));
  for (int i = 0; i < 4; ++i) {
    ARX_TRY(check_mat(out[i], i == 0));
    ARX_TRY(check_output(out[i], in, 4, i == 0 ? 1u : 0u));
    ARX_TRY(check_output(out[i], out, i, 0));
  }
  c.out = a->out, c.ldout = out[0].ld;
  c.z = a->z, c.ldz = out[1].ld;
  c.bias = a->bias;
  c.residual = a->residual, c.ldresidual = in[0].ld;
  c.act = a->act;
  if (copies) c.copies = a->copies;
  return launched(arx::launch_gemm(c, static_cast<cudaStream_t>(stream)), "arx_linear");
}

// dz [M][N rounded up to 8], then the partial sums of dbias.
size_t arx_linear_bwd_workspace_bytes(uint64_t M, uint64_t N) {
  if (M > kMaxDim || N > kMaxDim) return 0;
  return size_t(round16(M * ((N + 7) / 8 * 8) * 2) + arx::column_parts(M, N) * N * 4);
}

size_t arx_linear_bwd_copies_bytes(const arx_linear_bwd_args* a) {
  if (!a || a->M > kMaxDim || a->N > kMaxDim || a->K > kMaxDim) return 0;
  return backward_copies_bytes(*a);
}

arx_status arx_linear_bwd(const arx_linear_bwd_args* a, void* stream) {
  if (!a) return report(ARX_EINVAL, "null arguments");
  ARX_TRY(check_types(a->dtype, a->wdtype, false));
  ARX_TRY(check_dims(a->M, a->N, a->K));
  if (a->act < ARX_ACT_NONE || a->act > ARX_ACT_SILU) return report(ARX_EINVAL, "unknown activation %d", a->act);
  ARX_TRY(check_wait(a->wait_us));
  if (!a->dx && !a->dw && !a->dbias) return ok();
  const bool act = a->act != ARX_ACT_NONE, products = a->dx || a->dw;
  const Mat in[] = {mat("dout", a->dout, a->M, a->N, a->lddout, a->dtype),
                    mat("z", act ? a->z : nullptr, a->M, a->N, a->ldz, a->dtype),
                    mat("x", a->dw ? a->x : nullptr, a->M, a->K, a->ldx, a->dtype),
                    mat("w", a->dx ? a->w : nullptr, a->N, a->K, a->ldw, a->dtype)};
  const bool first_pass = (act && products) || a->dbias;
  const uint64_t need = first_pass ? arx_linear_bwd_workspace_bytes(a->M, a->N) : 0;
  const size_t copies = a->copies ? backward_copies_bytes(*a) : 0;
  ARX_TRY(check_copies(a->copies, a->copies_bytes, copies));
  const Mat out[] = {mat("dx", a->dx, a->M, a->K, a->lddx, a->dtype), mat("dw", a->dw, a->N, a->K, a->lddw, a->dtype),
                     vec("dbias", a->dbias, a->N, a->wdtype),
                     vec("workspace", a->workspace, a->workspace_bytes / 2, ARX_BF16),
                     vec("status", a->status, 1, ARX_F32), vec("copies", a->copies, copies / 2, ARX_BF16)};
  ARX_TRY(check_workspace(a->workspace, a->workspace_bytes, need));
  ARX_TRY(check_mat(in[0], true));
  ARX_TRY(check_mat(in[1], act));
  ARX_TRY(check_mat(in[2], a->dw != nullptr));
  ARX_TRY(check_mat(in[3], a->dx != nullptr));
  for (int i = 0; i < 6; ++i) {
    ARX_TRY(check_mat(out[i], false));
    ARX_TRY(check_output(out[i], in, 4, 0));
    ARX_TRY(check_output(out[i], out, i, 0));
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);

  // dz and dbias in one pass over dout.
  const void* dz = a->dout;
  uint64_t lddz = in[0].ld;
  uint8_t* ws = static_cast<uint8_t*>(a->workspace);
  const bool store = dz_in_workspace(*a);
  if ((first_pass || store) && a->N) {
    arx::ActGradCall g{};
    g.dout = a->dout, g.lddout = in[0].ld;
    g.rows = a->M, g.cols = a->N;
    if (act) g.z = a->z, g.ldz = in[1].ld;
    if (store) {
      lddz = g.lddz = (a->N + 7) / 8 * 8;
      dz = g.dz = ws;
    }
    g.dbias = a->dbias;
    g.part = reinterpret_cast<float*>(ws + round16(a->M * ((a->N + 7) / 8 * 8) * 2));
    g.act = a->act, g.dtype = a->dtype, g.wdtype = a->wdtype;
    const cudaError_t e = arx::launch_act_grad(g, units(in[0]) && units(in[1]), st);
    if (e != cudaSuccess) return launched(e, "arx_linear_bwd");
  }
  if (a->dx && a->M && a->K) {
    arx::GemmCall c = dx_product(*a, dz, lddz);
    c.out = a->dx, c.ldout = out[0].ld;
    if (copies) c.copies = a->copies;
    const cudaError_t e = arx::launch_gemm(c, st);
    if (e != cudaSuccess) return launched(e, "arx_linear_bwd");
  }
  if (a->dw && a->N && a->K) {  // its copies take the place of the other's, which have been read by then
    arx::GemmCall c = dw_product(*a, dz, lddz);
    c.out = a->dw, c.ldout = out[1].ld;
    if (copies) c.copies = a->copies;
    const cudaError_t e = arx::launch_gemm(c, st);
    if (e != cudaSuccess) return launched(e, "arx_linear_bwd");
  }
  return ok();
}

}  // extern "C"
